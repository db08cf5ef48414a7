"""GPU: attention with a shared prefix where a part holds many 128-token blocks
(rings that turn over, references that move, a second tile of rows, a tail in a
later block), and the join of more than 256 parts. The least workspace makes the
parts few; without it cases of this size are cut into single blocks."""
import numpy as np
import pytest
import torch

import transform_codec_b200 as kvc
from serving_ref import HostCache, attention, check_out
from test_gpu_attend import DT, _randn, i32

pytestmark = pytest.mark.gpu


def _part_bytes(rows, dim, parts):
    return (parts * rows * 4 + 15) // 16 * 16 + parts * rows * dim * 4


def _run(q, starts, prefix, share, host=None, parts=1):
    """parts: of the prefix."""
    n, Hq, D = q.shape
    seqs = len(starts) - 1
    att = kvc.Attention(q.dtype, Hq, prefix[0].shape[0], D, max_rows=n, max_seqs=seqs,
                        max_queries=max(b - a for a, b in zip(starts, starts[1:])),
                        max_kv=max(host.lens) if host else 1, prefix_tokens=prefix[0].shape[1])
    att._ws_bytes = min(att._ws_bytes, _part_bytes(n * Hq, D, parts + 1 if host else parts))
    out = torch.full((n, Hq, D), 5.0, dtype=q.dtype, device="cuda")
    lse = torch.full((n, Hq), 5.0, device="cuda")
    kw = {}
    if host is not None:
        kw.update(cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32(host.lens))
    att.run(q.cuda(), out, prefix=tuple(p.cuda() for p in prefix), prefix_len=i32(share), q_start=i32(starts),
            lse=lse, **kw)
    assert kvc.read_result(att.res) == (kvc.OK, 0)
    want, wl, tol = attention(q, starts, host, prefix, share, D ** -0.5)
    check_out(out, lse, want, wl, tol)


# factors of the keys along the prefix: scores as they come, growing, falling, one step up in a later block, waves
SHAPES = {
    "flat": lambda t: torch.ones(t),
    "growing": lambda t: torch.linspace(0, 8, t),
    "falling": lambda t: torch.linspace(8, 0, t),
    "step": lambda t: torch.where(torch.arange(t) < t * 2 // 3, 0.2, 9.0),
    "waves": lambda t: 4.0 * torch.sin(torch.arange(t) / 70.0),
}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs,group,queries,tokens", [
    (9, 4, 1, 1100),    # up to 128 rows: the same rows on alternate blocks, an odd number of them
    (16, 8, 1, 1024),   # exactly 128 rows, an even number of whole blocks
    (20, 4, 2, 1400),   # 160 rows: the second tile is partly empty
    (32, 8, 1, 896),    # two full tiles
    (11, 16, 2, 1153),  # two blocks of rows, one token in the last block
])
def test_many_blocks_a_part(shape, dt, dim, seqs, group, queries, tokens):
    """Shares that end in different blocks, at their borders, nowhere; the longest ends inside its block too."""
    prefix = [_randn(s, 1, tokens, dim, dt=DT[dt]) for s in (1, 2)]
    prefix[0] = (prefix[0].float() * SHAPES[shape](tokens)[:, None]).to(DT[dt])
    q = _randn(7, seqs * queries, group, dim, dt=DT[dt], spread=1.0)
    starts = list(range(0, seqs * queries + 1, queries))
    share = [(tokens, 0, 1, 640, 129, tokens - 3, 513, 512, 300)[i % 9] for i in range(seqs)]
    _run(q, starts, prefix, share)
    share = [min(n, tokens - 70) for n in share]
    for p in prefix:
        p[:, tokens - 70:] = float("nan")  # behind the longest share
    clean = [p.clone() for p in prefix]
    _run(q, starts, clean, share, parts=2)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("dim", [64, 128])
def test_many_blocks_and_a_cache(dt, dim):
    """Several heads, rows of two row blocks, three prefix parts of four blocks and the cache's part."""
    lens = [(i * 29) % 90 for i in range(24)]
    queries = [1 + i % 3 for i in range(24)]
    host = HostCache(kvc.CACHE_E2M1, 3, dim, 16, lens, seed=3)
    q = _randn(7, sum(queries), 3 * 8, dim, dt=DT[dt], spread=1.5)
    prefix = tuple(_randn(s, 3, 1500, dim, dt=DT[dt]) for s in (1, 2))
    share = [(1500, 1499, 0, 700, 130)[i % 5] for i in range(24)]
    for parts in (1, 3):
        _run(q, [0] + np.cumsum(queries).tolist(), prefix, share, host, parts)


@pytest.mark.parametrize("dim,group,queries", [(64, 2, 1), (128, 8, 1), (128, 4, 3)])
def test_join_of_more_than_256_parts(dim, group, queries):
    """One long sequence of one head."""
    n = 40001
    host = HostCache(kvc.CACHE_INT8, 1, dim, 64, [n], seed=5)
    q = _randn(6, queries, group, dim, dt=torch.float16, spread=1.0)
    prefix = tuple(_randn(s, 1, 400, dim, dt=torch.float16) for s in (1, 2))
    for p in (None, prefix):
        att = kvc.Attention(q.dtype, group, 1, dim, max_rows=queries, max_seqs=1, max_queries=queries, max_kv=n,
                            prefix_tokens=400 if p else 0)
        assert att._ws_bytes > _part_bytes(queries * group, dim, 256)
        out = torch.zeros(queries, group, dim, dtype=q.dtype, device="cuda")
        lse = torch.zeros(queries, group, device="cuda")
        att.run(q.cuda(), out, cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32([n]), lse=lse,
                q_start=i32([0, queries]), prefix=tuple(x.cuda() for x in p) if p else None)
        want, wl, tol = attention(q, [0, queries], host, p, None, dim ** -0.5)
        check_out(out, lse, want, wl, tol)
        assert kvc.read_result(att.res) == (kvc.OK, 0)


@pytest.mark.parametrize("queries", [1, 3])
def test_a_length_that_is_not_known(queries):
    """No max_kv given: long and short sequences, with and without a prefix."""
    lens = [9001, 5, 0]
    host = HostCache(kvc.CACHE_E4M3, 2, 128, 64, lens, seed=5)
    q = _randn(6, 3 * queries, 16, 128, dt=torch.bfloat16, spread=1.0)
    starts = [0, queries, 2 * queries, 3 * queries]
    prefix = tuple(_randn(s, 2, 200, 128, dt=torch.bfloat16) for s in (1, 2))
    for p in (None, prefix):
        att = kvc.Attention(q.dtype, 16, 2, 128, max_rows=3 * queries, max_seqs=3, max_queries=queries,
                            prefix_tokens=200 if p else 0)
        out = torch.zeros(3 * queries, 16, 128, dtype=q.dtype, device="cuda")
        lse = torch.zeros(3 * queries, 16, device="cuda")
        att.run(q.cuda(), out, cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32(lens), lse=lse,
                q_start=i32(starts), prefix=tuple(x.cuda() for x in p) if p else None)
        want, wl, tol = attention(q, starts, host, p, None, 128 ** -0.5)
        check_out(out, lse, want, wl, tol)


def test_large_prefix_values():
    """Values of 2^79 under weights that stay far above the reference: sums of P V within fp32."""
    tokens = 40000
    prefix = [_randn(s, 1, tokens, 64, dt=torch.bfloat16) for s in (1, 2)]
    prefix[1] = (prefix[1].float().clamp(-0.99, 0.99) * 2.0 ** 79).bfloat16()
    prefix[0][:] = 0
    prefix[0][:, 128:, 0] = 64 * 0.6931471805599453 / 8  # scores of 2^8 the first block's
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16)
    _run(q, [0, 1, 2], prefix, [tokens, tokens - 77])
