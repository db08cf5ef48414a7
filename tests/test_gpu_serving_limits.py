"""GPU: the serving calls at the largest counts that they accept, with layouts
that other tests do not use, and captured before anything else has run."""
import os
import subprocess
import sys

import pytest
import torch

import transform_codec_b200 as kvc
from serving_ref import FORMATS, HostCache, attention, check_out, quantise
from test_gpu_attend import _randn, i32

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_65535_sequences():
    """One token each: the answer is its value row, lse its score."""
    n, D = 65535, 64
    c = kvc.QuantCache(kvc.CACHE_INT8, 1, D, 16, n)
    k, v, q = (torch.randn(n, 1, D, device="cuda").bfloat16() for _ in range(3))
    table = torch.randperm(n, device="cuda", dtype=torch.int32)[:, None]
    kvc.cache_write(c, k, v, table[:, 0].long() * 16)
    kv = torch.zeros(2, 1, n, D, device="cuda")
    kvc.cache_read(c, table, torch.zeros(n, dtype=torch.int32, device="cuda"),
                   torch.arange(n + 1, dtype=torch.int32, device="cuda"), kv)
    att = kvc.Attention(torch.bfloat16, 1, 1, D, max_rows=n, max_seqs=n, max_kv=1)
    out, lse = torch.zeros_like(q), torch.zeros(n, 1, device="cuda")
    ones = torch.ones(n, dtype=torch.int32, device="cuda")
    for kw in ({}, dict(q_start=torch.arange(n + 1, dtype=torch.int32, device="cuda"))):
        out.zero_()
        att.run(q, out, cache=c, page_table=table, kv_len=ones, lse=lse, **kw)
        want = kv[1, 0]
        # the fp16 weight's step and the output's: 2^-11 and 2^-8 of the value, and fp32 steps
        assert ((out[:, 0].float() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -17)).all()
        score = (q[:, 0].double() * kv[0, 0].double()).sum(-1) / 8
        mag = (q[:, 0].double().abs() * kv[0, 0].double().abs()).sum(-1) / 8
        assert ((lse[:, 0].double() - score).abs() <= 2.0 ** -23 * (D + 8) * mag + 2.0 ** -18).all()
    assert kvc.read_result(att.res) == (kvc.OK, 0) and kvc.read_result(c.res) == (kvc.OK, 0)
    with pytest.raises(kvc.KvcError) as e:
        att.run(torch.cat((q, q[:1])), torch.cat((q, q[:1])), cache=c, page_table=torch.cat((table, table[:1])),
                kv_len=torch.cat((ones, ones[:1])))
    assert e.value.status == kvc.ERR_INVALID


@pytest.mark.parametrize("fmt", FORMATS)
def test_65535_heads(fmt):
    H, D = 65535, 64
    c = kvc.QuantCache(FORMATS[fmt], H, D, 16, 1)
    k, v = (_randn(s, 2, H, D, dt=torch.float16) for s in (1, 2))
    kvc.cache_write(c, k.cuda(), v.cuda(), torch.tensor([3, 4], device="cuda"))
    _, scales, _ = quantise(c.format, torch.stack((k, v), 1))
    assert torch.equal(c.scales[0, :, :, 3:5].cpu(), scales.permute(1, 2, 0))
    out = torch.zeros(2, H, 1, D, device="cuda")
    kvc.cache_read(c, i32([0])[None], i32([4]), i32([0, 1]), out)
    prefix = tuple(_randn(s, H, 2, D, dt=torch.float16) for s in (3, 4))
    q = _randn(5, 1, H, D, dt=torch.float16)
    # the cache's token 4 alone, at place 0 of a page of its own
    c2 = kvc.QuantCache(FORMATS[fmt], H, D, 16, 1)
    kvc.cache_write(c2, k[1:].cuda(), v[1:].cuda(), torch.tensor([0], device="cuda"))
    att = kvc.Attention(torch.float16, H, H, D, max_rows=1, max_seqs=1, max_kv=1, prefix_tokens=2)
    y = torch.zeros(1, H, D, dtype=torch.float16, device="cuda")
    att.run(q.cuda(), y, cache=c2, page_table=i32([0])[None], kv_len=i32([1]), prefix=tuple(p.cuda() for p in prefix))
    keys = torch.cat((prefix[0].double(), out[0].cpu().double()), 1)
    values = torch.cat((prefix[1].double(), out[1].cpu().double()), 1)
    p = torch.softmax(torch.einsum("hd,htd->ht", q[0].double(), keys) / 8, -1)
    want = torch.einsum("ht,htd->hd", p, values)
    # weights and outputs in fp16: 2^-11 each, the scores' fp32 sums and exponentials below that again
    bound = 2.0 ** -10 * torch.einsum("ht,htd->hd", p, values.abs()) + 2.0 ** -12 * want.abs() + 2.0 ** -24
    assert ((y[0].double().cpu() - want).abs() <= bound).all()
    assert kvc.read_result(att.res) == (kvc.OK, 0)


def test_shared_queries_and_head_major_outputs():
    """One query row for the whole batch (a stride of zero), keys and values of one row for all tokens, out as
    [head][row]."""
    host = HostCache(kvc.CACHE_E4M3, 2, 64, 16, [70, 9, 33], seed=2)
    one = _randn(3, 1, 8, 64, dt=torch.bfloat16)
    out = torch.zeros(8, 3, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    prefix = tuple(_randn(s, 2, 140, 64, dt=torch.bfloat16) for s in (1, 2))
    att = kvc.Attention(torch.bfloat16, 8, 2, 64, max_rows=3, max_seqs=3, max_kv=70, prefix_tokens=140)
    att.run(one.cuda().expand(3, 8, 64), out, cache=host.gpu(), page_table=host.table.cuda(), kv_len=i32(host.lens),
            prefix=tuple(p.cuda() for p in prefix))
    want, lse, tol = attention(one.expand(3, 8, 64), [0, 1, 2, 3], host, prefix, None, 64 ** -0.5)
    check_out(out, None, want, lse, tol)
    c = kvc.QuantCache(kvc.CACHE_E2M1, 2, 64, 16, 3)
    k = _randn(3, 1, 1, 64, dt=torch.float32)
    kvc.cache_write(c, k.cuda().expand(40, 2, 64), -k.cuda().expand(40, 2, 64), torch.arange(40, device="cuda"))
    _, scales, _ = quantise(c.format, torch.stack((k, -k), 1)[0, :, 0])
    rows = c.scales.cpu().permute(1, 2, 0, 3).reshape(2, 2, 48)[:, :, :40]
    assert torch.equal(rows, scales[:, None, None].expand(2, 2, 40))


FIRST = r"""
import sys
import torch
sys.path.insert(0, ROOT)
import transform_codec_b200 as kvc
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
g = torch.Generator(device="cuda").manual_seed(1)
rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
k, v, pk, pv, q = rnd(40, 2, 128), rnd(40, 2, 128), rnd(2, 500, 128), rnd(2, 500, 128), rnd(2, 16, 128)
slots, table, lens = torch.arange(40, device="cuda"), i32(0, 1, 1, 2).reshape(2, 2), i32(20, 24)
cache = kvc.QuantCache(kvc.CACHE_E4M3, 2, 128, 16, 3)
att = kvc.Attention(torch.bfloat16, 16, 2, 128, max_rows=2, max_seqs=2, max_kv=24, prefix_tokens=500)
out, back = torch.zeros_like(q), torch.zeros(2, 2, 24, 128, device="cuda")
args = table[1:].contiguous(), i32(0), i32(0, 24)
def step():
    kvc.cache_write(cache, k, v, slots)
    att.run(q, out, cache=cache, page_table=table, kv_len=lens, prefix=(pk, pv))
    kvc.cache_read(cache, *args, back)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):  # the library's first calls of this process
    step()
graph.replay()
torch.cuda.synchronize()
first = out.clone(), back.clone()
assert first[0].abs().max() > 0 and first[1].abs().max() > 0
for t in (out, back, cache.codes, cache.scales):
    t.zero_()
step()
torch.cuda.synchronize()
assert torch.equal(out, first[0]) and torch.equal(back, first[1])
assert kvc.read_result(att.res)[0] == kvc.OK and kvc.read_result(cache.res)[0] == kvc.OK
print("first-child: ok")
"""


def test_the_first_calls_may_be_captured():
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + FIRST], capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "first-child: ok" in r.stdout
