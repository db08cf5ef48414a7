"""GPU: attention reports query starts that are out of range or out of order,
whether or not a row lies in them."""
import pytest
import torch

import transform_codec_b200 as kvc
from serving_ref import HostCache
from test_gpu_attend import _randn, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_cache", [False, True])
@pytest.mark.parametrize("q_start,same", [
    ((0, 2, 5), [0, 1]),     # the second sequence's rows do not exist
    ((0, 2, 1, 2), [0]),     # descending
    ((-1, 1, 2), [1]),
    ((0, 1, -7, 2), []),
    ((0, 2, 2, 3), [0, 1]),
])
def test_attention_reports_bad_query_starts(with_cache, q_start, same):
    n = len(q_start) - 1
    host = HostCache(kvc.CACHE_INT8, 1, 64, 16, [40] * n, seed=2)
    q = _randn(3, 2, 4, 64, dt=torch.bfloat16).cuda()
    prefix = tuple(_randn(s, 1, 200, 64, dt=torch.bfloat16).cuda() for s in (1, 2))
    att = kvc.Attention(q.dtype, 4, 1, 64, max_rows=2, max_seqs=n, max_queries=2, max_kv=40, prefix_tokens=200)
    kw = dict(cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32(host.lens)) if with_cache else {}
    if not with_cache:
        ok = torch.zeros_like(q)
        att.run(q, ok, prefix=prefix)  # all of the prefix for every row
        assert kvc.read_result(att.res)[0] == kvc.OK
    out = torch.full_like(q, 5.0)
    att.run(q, out, prefix=prefix, q_start=i32(q_start), **kw)
    assert kvc.read_result(att.res)[0] == kvc.ERR_INVALID
    if not with_cache:
        assert torch.equal(out[same], ok[same])


def test_attention_over_a_prefix_accepts_good_starts():
    q = _randn(3, 6, 4, 64, dt=torch.bfloat16).cuda()
    prefix = tuple(_randn(s, 1, 200, 64, dt=torch.bfloat16).cuda() for s in (1, 2))
    for starts in ((0, 6), (0, 0, 3, 3, 6, 6), (2, 4), [0] * 700 + [6]):
        att = kvc.Attention(q.dtype, 4, 1, 64, max_rows=6, max_seqs=len(starts) - 1, max_queries=6, prefix_tokens=200)
        att.run(q, torch.zeros_like(q), prefix=prefix, q_start=i32(starts))
        assert kvc.read_result(att.res)[0] == kvc.OK


@pytest.mark.parametrize("with_cache", [False, True])
@pytest.mark.parametrize("share", [(201, 200, 0), (200, -1, 0), (200, 200, 201), (0, 0, -5)])
def test_attention_reports_bad_shares_of_sequences_without_rows(with_cache, share):
    host = HostCache(kvc.CACHE_INT8, 1, 64, 16, [40] * 3, seed=2)
    q = _randn(3, 2, 4, 64, dt=torch.bfloat16).cuda()
    prefix = tuple(_randn(s, 1, 200, 64, dt=torch.bfloat16).cuda() for s in (1, 2))
    att = kvc.Attention(q.dtype, 4, 1, 64, max_rows=2, max_seqs=3, max_queries=2, max_kv=40, prefix_tokens=200)
    kw = dict(cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32(host.lens)) if with_cache else {}
    empty = next(i for i, n in enumerate(share) if not 0 <= n <= 200)
    starts = [0] * (empty + 2) + [2] * (2 - empty)  # sequence `empty` has no rows
    out = torch.zeros_like(q)
    att.run(q, out, prefix=prefix, q_start=i32(starts), prefix_len=i32([200] * 3), **kw)
    assert kvc.read_result(att.res)[0] == kvc.OK
    att.run(q, out, prefix=prefix, q_start=i32(starts), prefix_len=i32(share), **kw)
    assert kvc.read_result(att.res)[0] == kvc.ERR_INVALID


def test_empty_steps():
    """No rows, and sequences without any: nothing is written and nothing refused."""
    host = HostCache(kvc.CACHE_INT8, 1, 64, 16, [40], seed=2)
    c = host.gpu()
    prefix = tuple(_randn(s, 1, 200, 64, dt=torch.bfloat16).cuda() for s in (1, 2))
    att = kvc.Attention(torch.bfloat16, 4, 1, 64, max_rows=2, max_seqs=2, max_kv=40, prefix_tokens=200)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(0, 3, dtype=torch.int32, device="cuda"), i32([])
    for kw in (dict(cache=c, page_table=table, kv_len=lens), dict(prefix=prefix), dict(prefix=prefix, prefix_len=lens),
               dict(cache=c, page_table=table, kv_len=lens, prefix=prefix, q_start=i32([0])),
               dict(cache=c, page_table=host.table.cuda(), kv_len=i32([40]), q_start=i32([0, 0]))):
        att.run(q, q.clone(), lse=torch.zeros(0, 4, device="cuda"), **kw)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 5.0)
    att.run(q, out, cache=c, page_table=table, kv_len=lens, q_start=i32([0]))
    assert (out == 5.0).all() and kvc.read_result(att.res)[0] == kvc.OK
