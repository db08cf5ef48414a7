"""GPU: attention over the serving cache and a shared prefix against fp64."""
import numpy as np
import pytest
import torch

import kvgen
import transform_codec_b200 as kvc
from serving_ref import FORMATS, HostCache, attention, check_out

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _randn(seed, *shape, dt=torch.float32, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * spread).to(dt)


def _run(host, q, starts, prefix=None, prefix_len=None, scale=None, with_lse=True, max_queries=None, max_kv=None,
         att=None, check=True):
    """One call, with two rows before the first sequence's and three behind the last that must stay as they are."""
    n, Hq, D = q.shape
    H = host.heads if host is not None else prefix[0].shape[0]
    scale = D ** -0.5 if scale is None else scale
    seqs = len(starts) - 1
    if att is None:
        att = kvc.Attention(q.dtype, Hq, H, D, max_rows=n + 5, max_seqs=seqs,
                            max_queries=max_queries or max([1] + [b - a for a, b in zip(starts, starts[1:])]),
                            max_kv=max_kv if max_kv is not None else (max(host.lens) if host is not None else 0),
                            prefix_tokens=0 if prefix is None else prefix[0].shape[1])
    qg = torch.zeros(n + 5, Hq, D, dtype=q.dtype, device="cuda")
    qg[2:2 + n] = q.cuda()
    out = torch.full((n + 5, Hq, D), 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full((n + 5, Hq), 5.0, device="cuda") if with_lse else None
    kw = dict(q_start=i32(s + 2 for s in starts), scale=scale, lse=lse)
    if host is not None:
        kw.update(cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32(host.lens))
    if prefix is not None:
        kw.update(prefix=(prefix[0].cuda(), prefix[1].cuda()))
        if prefix_len is not None:
            kw.update(prefix_len=i32(prefix_len))
    att.run(qg, out, **kw)
    assert kvc.read_result(att.res) == (kvc.OK, 0)
    assert (out[:2] == 5.0).all() and (out[2 + n:] == 5.0).all()
    if with_lse:
        assert (lse[:2] == 5.0).all() and (lse[2 + n:] == 5.0).all()
        lse = lse[2:2 + n]
    out = out[2:2 + n]
    if check:
        want, wl, tol = attention(q, starts, host, prefix, prefix_len, scale)
        check_out(out, lse, want, wl, tol)
    return out, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,page,lens", [
    (1, 1, 16, [1]), (2, 8, 16, [15, 16, 17, 0, 33]), (3, 7, 32, [63, 64, 65]), (8, 4, 64, [300, 1, 129]),
    (1, 16, 128, [700]), (2, 3, 1024, [1025, 5]),
])
def test_single_queries_over_the_cache(fmt, dt, dim, heads, group, page, lens):
    host = HostCache(FORMATS[fmt], heads, dim, page, lens, seed=len(lens))
    q = _randn(3, len(lens), heads * group, dim, dt=DT[dt], spread=1.5)
    _run(host, q, list(range(len(lens) + 1)))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("dim,heads,group,page,lens,queries", [
    (128, 2, 8, 16, [100, 3, 0, 40, 7], [4, 5, 2, 0, 7]),  # more queries than tokens: the first rows see nothing
    (64, 1, 5, 16, [50, 200], [3, 9]),
    (128, 1, 16, 64, [90, 64, 63], [8, 1, 6]),
    (64, 4, 1, 32, [33, 31], [33, 40]),
])
def test_several_queries_a_sequence(fmt, dt, dim, heads, group, page, lens, queries):
    host = HostCache(FORMATS[fmt], heads, dim, page, lens, seed=7)
    q = _randn(4, sum(queries), heads * group, dim, dt=DT[dt], spread=1.5)
    _run(host, q, [0] + np.cumsum(queries).tolist())


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_sequences_are_split(fmt):
    host = HostCache(FORMATS[fmt], 1, 128, 64, [9001, 40, 4096], seed=8)
    q = _randn(5, 3, 8, 128, dt=torch.float16, spread=2.0)
    _run(host, q, [0, 1, 2, 3])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group,rows,tokens", [
    (1, 1, 1, 1), (2, 1, 3, 2), (1, 8, 5, 127), (2, 4, 20, 128), (1, 3, 43, 129), (2, 16, 9, 255), (1, 8, 33, 1000),
    (3, 2, 70, 300), (1, 16, 40, 513),
])
def test_prefix_alone(dt, dim, heads, group, rows, tokens):
    q = _randn(6, rows, heads * group, dim, dt=DT[dt], spread=1.5)
    prefix = tuple(_randn(s, heads, tokens, dim, dt=DT[dt]) for s in (1, 2))
    lens = [tokens] * rows
    att_starts = list(range(rows + 1))
    _run(None, q, att_starts, prefix, lens)
    _run(None, q, [0, rows], prefix)  # one sequence of all the rows, nothing masked


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("dim", [64, 128])
def test_prefix_lengths_differ(dt, dim):
    """Sequences that share none, one token, parts that end inside and at a tile's border, or all of the prefix."""
    lens = [0, 1, 127, 128, 129, 400, 64, 0, 256, 257, 399]
    n = len(lens)
    prefix = tuple(_randn(s, 2, 400, dim, dt=DT[dt]) for s in (1, 2))
    q = _randn(7, 2 * n, 2 * 4, dim, dt=DT[dt], spread=1.5)
    _run(None, q, list(range(0, 2 * n + 1, 2)), prefix, lens)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("dim,heads,group,page,tokens,lens,queries", [
    (128, 2, 8, 16, 300, [20, 0, 5, 77], [1, 1, 1, 1]),
    (64, 3, 1, 16, 130, [0, 16, 3], [2, 1, 4]),
    (128, 1, 4, 64, 2049, [65, 200] * 20, [1, 2] * 20),
    (128, 4, 16, 32, 64, [1, 31, 33, 0, 2], [1, 3, 1, 1, 2]),
])
def test_prefix_and_cache_join(fmt, dt, dim, heads, group, page, tokens, lens, queries):
    host = HostCache(FORMATS[fmt], heads, dim, page, lens, seed=9)
    q = _randn(8, sum(queries), heads * group, dim, dt=DT[dt], spread=1.5)
    prefix = tuple(_randn(s, heads, tokens, dim, dt=DT[dt]) for s in (1, 2))
    starts = [0] + np.cumsum(queries).tolist()
    _run(host, q, starts, prefix)
    share = [(tokens * (i % 4)) // 3 for i in range(len(lens))]
    _run(host, q, starts, prefix, share, with_lse=False)


def test_rows_that_see_nothing():
    """No prefix tokens and no cache tokens: zeros and -infinity, next to rows that see some."""
    host = HostCache(kvc.CACHE_E4M3, 2, 128, 16, [0, 3, 0], seed=1)
    q = _randn(1, 9, 16, 128, dt=torch.bfloat16)
    prefix = tuple(_randn(s, 2, 50, 128, dt=torch.bfloat16) for s in (1, 2))
    out, lse = _run(host, q, [0, 2, 7, 9], prefix, [0, 0, 9])
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    assert (out[2:4] == 0).all() and torch.isneginf(lse[2:4]).all()  # five queries, three tokens
    out, lse = _run(host, q, [0, 2, 7, 9])
    assert (out[7:] == 0).all() and torch.isneginf(lse[7:]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_scores_far_apart(fmt):
    """Scores in the hundreds, growing and falling along the sequence, and values of very different sizes."""
    host = HostCache(FORMATS[fmt], 1, 128, 16, [400, 400], seed=3, spread=2.5)
    for b in range(2):
        pos = torch.arange(400)
        page, at = host.table[b].long()[pos // 16], pos % 16
        ramp = torch.linspace(0.01, 4.0, 400)
        host.scales[page, 0, :, at] *= (ramp if b == 0 else ramp.flip(0))[:, None]
    q = _randn(2, 2, 8, 128, dt=torch.float16, spread=1.0)
    prefix = (_randn(1, 1, 300, 128, dt=torch.float16, spread=1.0) * torch.linspace(0, 6, 300)[:, None].half(),
              _randn(2, 1, 300, 128, dt=torch.float16))
    _run(host, q, [0, 1, 2])
    _run(host, q, [0, 1, 2], prefix)
    _run(None, q, [0, 1, 2], tuple(p.flip(1).contiguous() for p in prefix))


def test_values_of_zero_and_of_a_tiny_row():
    """Rows whose values are all zero (scale 0) or tiny take their share of the softmax."""
    host = HostCache(kvc.CACHE_INT8, 1, 64, 16, [40], seed=4)
    pos = torch.arange(40)
    page, at = host.table[0].long()[pos // 16], pos % 16
    host.scales[page[3:9], 1, :, at[3:9]] = 0.0
    host.codes[page[3:9], 1, :, at[3:9]] = 0
    host.scales[page[20], 1, :, at[20]] = 2.0 ** -90
    q = _randn(5, 1, 4, 64, dt=torch.bfloat16, spread=1.5)
    _run(host, q, [0, 1])
    host.scales[page, 1, :, at] = 0.0
    host.codes[page, 1, :, at] = 0
    out, _ = _run(host, q, [0, 1])
    assert (out == 0).all()


@pytest.mark.parametrize("kv", [0, 1])
def test_nan_rows_reach_those_who_see_them(kv):
    host = HostCache(kvc.CACHE_E2M1, 1, 64, 16, [40, 40], seed=5)
    p = int(host.table[0, 1])
    host.scales[p, kv, :, 3] = float("nan")  # token 19 of sequence 0
    q = _randn(5, 4, 4, 64, dt=torch.bfloat16)
    out, lse = _run(host, q, [0, 2, 4], check=False)
    assert torch.isnan(out[:2]).all() and torch.isfinite(out[2:]).all()
    assert torch.isnan(lse[:2]).all() if kv == 0 else torch.isfinite(lse).all()  # values have no part in lse
    host.lens[0] = 20  # seen by the last of two queries alone
    out, _ = _run(host, q, [0, 2, 4], check=False)
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all()


def test_prefix_nan_beyond_a_sequence_s_share_is_not_seen():
    prefix = [_randn(s, 1, 300, 128, dt=torch.bfloat16) for s in (1, 2)]
    q = _randn(5, 3, 8, 128, dt=torch.bfloat16)
    clean = _run(None, q, [0, 1, 2, 3], prefix, [150, 150, 0])[0].clone()
    dirty = [p.clone() for p in prefix]
    for p in dirty:
        p[:, 150:] = float("nan")
    dirty[0][:, 200:] = float("inf")
    out, _ = _run(None, q, [0, 1, 2, 3], dirty, [150, 150, 0], check=False)
    assert torch.equal(out, clean)


def test_a_sequence_s_share_hides_what_others_see():
    """A NaN that one sequence's share of the prefix holds stays out of a shorter share's rows."""
    prefix = [_randn(s, 1, 300, 128, dt=torch.float16) for s in (1, 2)]
    q = _randn(5, 2, 8, 128, dt=torch.float16)
    clean = _run(None, q, [0, 1, 2], prefix, [150, 300])[0].clone()
    prefix[0][:, 170] = float("nan")
    out, _ = _run(None, q, [0, 1, 2], prefix, [150, 300], check=False)
    assert torch.equal(out[0], clean[0]) and torch.isnan(out[1]).all()


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-40, 3.0])
def test_unusual_scales(scale):
    """Negative scales turn the order round, a scale of zero weighs all tokens alike."""
    host = HostCache(kvc.CACHE_E2M1, 2, 128, 16, [50, 3], seed=2)
    q = _randn(3, 5, 8, 128, dt=torch.float16, spread=0.5)
    prefix = tuple(_randn(s, 2, 200, 128, dt=torch.float16) for s in (1, 2))
    _run(host, q, [0, 4, 5], prefix, [130, 0], scale=scale)
    _run(host, q, [0, 4, 5], scale=scale)


def test_prefix_that_no_one_shares():
    q = _randn(5, 3, 8, 128, dt=torch.bfloat16)
    prefix = tuple(_randn(s, 1, 300, 128, dt=torch.bfloat16) for s in (1, 2))
    out, lse = _run(None, q, [0, 1, 2, 3], prefix, [0, 0, 0])
    assert (out == 0).all() and torch.isneginf(lse).all()
    q = _randn(5, 100, 8, 128, dt=torch.bfloat16)  # more rows than one block takes
    out, lse = _run(None, q, [0, 50, 100], prefix, [0, 0])
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_queries_that_are_not_finite_stay_in_their_rows(what):
    host = HostCache(kvc.CACHE_E4M3, 1, 128, 16, [70, 5], seed=2)
    prefix = tuple(_randn(s, 1, 200, 128, dt=torch.bfloat16) for s in (1, 2))
    q = _randn(3, 2, 8, 128, dt=torch.bfloat16)
    for kw in (dict(host=host), dict(host=None, prefix=prefix), dict(host=host, prefix=prefix)):
        clean, _ = _run(q=q, starts=[0, 1, 2], **kw)
        bad = q.clone()
        bad[0, 3, 17] = what
        out, lse = _run(q=bad, starts=[0, 1, 2], check=False, **kw)
        assert torch.isnan(out[0, 3]).all()
        keep = torch.ones(2, 8, dtype=torch.bool)
        keep[0, 3] = False
        assert torch.equal(out[keep.cuda()], clean[keep.cuda()])


def test_zero_queries_weigh_all_tokens_alike():
    host = HostCache(kvc.CACHE_INT8, 2, 64, 16, [33], seed=2)
    _run(host, torch.zeros(1, 4, 64, dtype=torch.float16), [0, 1])


def test_large_and_tiny_queries():
    """Magnitudes near bf16's ends: the score's scale is kept apart from the elements."""
    host = HostCache(kvc.CACHE_INT8, 1, 64, 16, [40], seed=2)
    for size in (2.0 ** 100, 2.0 ** -100):
        q = _randn(3, 1, 4, 64, dt=torch.bfloat16) * size
        _run(host, q, [0, 1], scale=1.0 / size)


def test_many_sequences():
    """More sequences than any one wave of blocks, most of them short, some empty."""
    lens = [(i * 37) % 90 for i in range(700)]
    host = HostCache(kvc.CACHE_E4M3, 1, 64, 16, lens, seed=2)
    q = _randn(3, 700, 2, 64, dt=torch.bfloat16)
    _run(host, q, list(range(701)))
    prefix = tuple(_randn(s, 1, 140, 64, dt=torch.bfloat16) for s in (1, 2))
    _run(host, q, list(range(701)), prefix, [(i * 13) % 141 for i in range(700)])


@pytest.mark.parametrize("fmt", FORMATS)
def test_hints_and_workspace_do_not_change_results_beyond_rounding(fmt):
    """Wrong expectations of the largest sequence, and the least workspace."""
    lens, queries = [500, 2000, 30], [3, 1, 6]
    host = HostCache(FORMATS[fmt], 2, 64, 32, lens, seed=6)
    q = _randn(6, 10, 8, 64, dt=torch.float16, spread=1.5)
    prefix = tuple(_randn(s, 2, 700, 64, dt=torch.float16) for s in (1, 2))
    for mq, mk in ((1, 1), (1, 100000), (64, 2000)):
        _run(host, q, [0, 3, 4, 10], prefix, max_queries=mq, max_kv=mk)
        _run(host, q, [0, 3, 4, 10], max_queries=mq, max_kv=mk)
    att = kvc.Attention(q.dtype, 8, 2, 64, max_rows=15, max_seqs=3, max_queries=6, max_kv=2000, prefix_tokens=700)
    least = kvc.lib().kvc_attend_workspace_min(att._ref)
    assert 0 < least <= att._ws_bytes
    att._ws_bytes = least
    _run(host, q, [0, 3, 4, 10], prefix, att=att)
    att._ws_bytes = least - 1
    with pytest.raises(kvc.KvcError) as e:
        _run(host, q, [0, 3, 4, 10], prefix, att=att)
    assert e.value.status == kvc.ERR_CAPACITY


def test_strided_queries_and_outputs():
    """q as a part of a fused projection, out as a part of a wider buffer, prefix as slices of a larger cache."""
    host = HostCache(kvc.CACHE_E4M3, 2, 64, 16, [70, 9], seed=2)
    Hq, D = 6, 64
    fused = _randn(3, 2, Hq + 4, D, dt=torch.bfloat16)
    q = fused[:, 1:1 + Hq]
    cache = _randn(4, 2, 2, 2, 150, D, dt=torch.bfloat16).cuda()  # [layer][k/v][head][token][channel]
    pk, pv = cache[1, 0, :, :130], cache[1, 1, :, :130]
    wide = torch.full((2, Hq, 3 * D), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :, D:2 * D]
    att = kvc.Attention(q.dtype, Hq, 2, D, max_rows=2, max_seqs=2, max_kv=70, prefix_tokens=130)
    g = fused.cuda()
    att.run(g[:, 1:1 + Hq], out, cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32(host.lens),
            prefix=(pk, pv))
    want, lse, tol = attention(q, [0, 1, 2], host, (pk.cpu(), pv.cpu()), None, D ** -0.5)
    check_out(out, None, want, lse, tol)
    assert (wide[:, :, :D] == 5.0).all() and (wide[:, :, 2 * D:] == 5.0).all()


def test_bad_device_indices_set_the_status():
    host = HostCache(kvc.CACHE_INT8, 1, 64, 16, [40, 30], seed=2)
    q = _randn(3, 2, 4, 64, dt=torch.bfloat16).cuda()
    prefix = tuple(_randn(s, 1, 60, 64, dt=torch.bfloat16).cuda() for s in (1, 2))
    c = host.gpu()
    out = torch.zeros_like(q)
    att = kvc.Attention(q.dtype, 4, 1, 64, max_rows=2, max_seqs=2, max_kv=40, prefix_tokens=60)
    good = dict(page_table=host.table.cuda(), kv_len=i32(host.lens), prefix_len=i32([60, 10]))
    att.run(q, out, cache=c, prefix=prefix, **good)
    assert kvc.read_result(att.res)[0] == kvc.OK
    ok = out.clone()
    table = host.table.clone()
    table[0, 2] = c.n_pages
    for change in (dict(page_table=table.cuda()), dict(kv_len=i32([10 ** 6, 30])), dict(kv_len=i32([-1, 30])),
                   dict(prefix_len=i32([61, 10])), dict(prefix_len=i32([-1, 10])),
                   dict(q_start=i32([0, 1, 5])), dict(q_start=i32([-3, 1, 2]))):
        att.res.zero_()
        att.run(q, out, cache=c, prefix=prefix, **{**good, **change})
        assert kvc.read_result(att.res)[0] == kvc.ERR_INVALID, change
        other = 0 if change.get("q_start") is not None and int(change["q_start"][0]) == 0 else 1
        assert torch.equal(out[other], ok[other])  # the other sequence is answered as before


def test_other_streams_and_graphs():
    """Two Attention objects at once on two streams, and a captured step replayed on new contents and lengths."""
    hosts = [HostCache(kvc.CACHE_E4M3, 2, 128, 16, [600, 35], seed=s) for s in (1, 2)]
    qs = [_randn(s, 2, 8, 128, dt=torch.bfloat16, spread=1.5) for s in (3, 4)]
    prefix = tuple(_randn(s, 2, 500, 128, dt=torch.bfloat16) for s in (1, 2))
    gp = tuple(p.cuda() for p in prefix)
    caches = [h.gpu() for h in hosts]
    tables = [h.table.cuda() for h in hosts]
    lens = [i32(h.lens) for h in hosts]
    q = [x.cuda() for x in qs]
    outs = [torch.zeros_like(x) for x in q]
    atts = [kvc.Attention(torch.bfloat16, 8, 2, 128, max_rows=2, max_seqs=2, max_kv=600, prefix_tokens=500)
            for _ in hosts]
    streams = [torch.cuda.Stream() for _ in hosts]
    torch.cuda.synchronize()
    for _ in range(20):
        for j in range(2):
            atts[j].run(q[j], outs[j], cache=caches[j], page_table=tables[j], kv_len=lens[j], prefix=gp,
                        stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        want, lse, tol = attention(qs[j], [0, 1, 2], hosts[j], prefix, None, 128 ** -0.5)
        check_out(outs[j], None, want, lse, tol)
    # a step: write the new tokens' keys and values, attend over them
    j = 0
    k, v = (torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.full((2,), -1, dtype=torch.int64, device="cuda")

    def step():
        kvc.cache_write(caches[j], k, v, slots)
        atts[j].run(q[j], outs[j], cache=caches[j], page_table=tables[j], kv_len=lens[j], prefix=gp)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    host = hosts[0]
    for t in range(3):  # the second sequence grows by a token a step
        host.lens[1] += 1
        pos = host.lens[1] - 1
        new = [_randn(50 + 2 * t + e, 2, 2, 128, dt=torch.bfloat16) for e in range(2)]
        k.copy_(new[0])
        v.copy_(new[1])
        slots.copy_(torch.tensor([-1, int(host.table[1, pos // 16]) * 16 + pos % 16]))
        lens[0].copy_(i32(host.lens))
        qs[0] = _randn(90 + t, 2, 8, 128, dt=torch.bfloat16, spread=1.5)
        q[0].copy_(qs[0])
        graph.replay()
        torch.cuda.synchronize()
        host.codes, host.scales = caches[0].codes.cpu(), caches[0].scales.cpu()
        want, lse, tol = attention(qs[0], [0, 1, 2], host, prefix, None, 128 ** -0.5)
        check_out(outs[0], None, want, lse, tol)
    assert kvc.read_result(atts[0].res)[0] == kvc.OK and kvc.read_result(caches[0].res)[0] == kvc.OK


def test_same_inputs_same_bits():
    """No result depends on the order in which blocks run."""
    host = HostCache(kvc.CACHE_INT8, 2, 128, 16, [3000, 100, 0, 777], seed=2)
    q = _randn(3, 4, 16, 128, dt=torch.float16, spread=1.5)
    prefix = tuple(_randn(s, 2, 1500, 128, dt=torch.float16) for s in (1, 2))
    first, l1 = _run(host, q, [0, 1, 2, 3, 4], prefix, check=False)
    for _ in range(5):
        out, l2 = _run(host, q, [0, 1, 2, 3, 4], prefix, check=False)
        assert torch.equal(out, first) and torch.equal(l1, l2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_from_container_to_answers_and_back(fmt):
    """An exported cache comes out of its container as the prefix that a batch shares; the batch's own tokens are
    written to the quantised cache, attended to, read back as slices and coded into a container again."""
    w = kvgen.Workload("serving", "lossless", kvgen.BF16, 1, 2, 300, 128, 0.9, 1e4)
    x = kvgen.slices(w)  # [2 * heads][tokens][dim] bf16 bits
    plan = kvc.Plan(kvc.Shape.from_workload(w))
    codec = kvc.Codec(plan, kvc.LOSSLESS, w.n_slices)
    src = torch.from_numpy(x.view(np.int16).ravel()).cuda()
    st, nbytes = kvc.read_result(codec.encode(src))
    assert st == kvc.OK
    st, _ = kvc.read_result(codec.decode(codec.container, nbytes))
    assert st == kvc.OK
    slices = codec.decoded[:x.size].view(torch.bfloat16).reshape(2, 2, 300, 128)
    prefix = (slices[0], slices[1])
    # five sequences write 1 .. 40 tokens of their own
    lens, page = [40, 1, 17, 16, 5], 16
    need = [-(-n // page) for n in lens]
    cache = kvc.QuantCache(FORMATS[fmt], 2, 128, page, sum(need))
    table = torch.full((5, 3), -1, dtype=torch.int32)
    slots, at = [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = torch.arange(at, at + need[b])
        slots += [at * page + t for t in range(n)]
        at += need[b]
    k, v = (_randn(s, sum(lens), 2, 128, dt=torch.bfloat16) for s in (5, 6))
    kvc.cache_write(cache, k.cuda(), v.cuda(), torch.tensor(slots, device="cuda"))
    q = _randn(7, 5, 16, 128, dt=torch.bfloat16, spread=0.5)
    out = torch.zeros(5, 16, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(5, 16, device="cuda")
    att = kvc.Attention(torch.bfloat16, 16, 2, 128, max_rows=5, max_seqs=5, max_kv=40, prefix_tokens=300)
    att.run(q.cuda(), out, cache=cache, page_table=table.cuda(), kv_len=i32(lens), prefix=prefix, lse=lse)
    host = HostCache.__new__(HostCache)
    host.fmt, host.heads, host.dim, host.page, host.lens, host.table = FORMATS[fmt], 2, 128, page, lens, table
    host.codes, host.scales = cache.codes.cpu(), cache.scales.cpu()
    host.micro = None if cache.micro is None else cache.micro.cpu()
    want, wl, tol = attention(q, list(range(6)), host, tuple(p.cpu() for p in prefix), None, 128 ** -0.5)
    check_out(out, lse, want, wl, tol)
    # sequence 0 leaves as a container
    back = torch.zeros(2, 2, 40, 128, dtype=torch.bfloat16, device="cuda")
    kvc.cache_read(cache, table[:1].cuda(), i32([0]), i32([0, 40]), back)
    plan40 = kvc.Plan(kvc.Shape(kvc.BF16, 1, 2, 40, 128))
    c40 = kvc.Codec(plan40, kvc.LOSSLESS, 4)
    st, nbytes = kvc.read_result(c40.encode(back))
    assert st == kvc.OK
    st, _ = kvc.read_result(c40.decode(c40.container, nbytes))
    assert st == kvc.OK
    assert torch.equal(c40.decoded[:back.numel()].view(torch.bfloat16).reshape(back.shape), back)
    assert kvc.read_result(att.res)[0] == kvc.OK and kvc.read_result(cache.res)[0] == kvc.OK
