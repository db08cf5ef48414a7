"""The shared-prefix kernel's waits are bounded: with the "wait0" test build
(every wait gives up without polling; the drain waits keep their long bound, so
copies and products have ended before the block leaves) a call reports
KVC_ERR_TIMEOUT in its sticky result and the context stays usable. Nothing
faults. The build runs in a child process, since a process loads one libkvc."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import torch
sys.path.insert(0, ROOT)
import transform_codec_b200 as kvc
assert kvc.LIB_PATH.endswith("libkvc_wait0.so"), kvc.LIB_PATH
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
cache = kvc.QuantCache(kvc.CACHE_INT8, 2, 128, 16, 4)
k, v = (torch.randn(2, 2, 128, device="cuda").bfloat16() for _ in range(2))
kvc.cache_write(cache, k, v, torch.tensor([0, 16], device="cuda"))
q = torch.randn(2, 16, 128, device="cuda").bfloat16()
out = torch.zeros_like(q)
table = i32(0, 1).reshape(2, 1)
for tokens in (100, 2000):
    prefix = tuple(torch.randn(2, tokens, 128, device="cuda").bfloat16() for _ in range(2))
    att = kvc.Attention(torch.bfloat16, 16, 2, 128, max_rows=2, max_seqs=2, max_kv=1, prefix_tokens=tokens)
    for _ in range(2):
        att.res.zero_()
        att.run(q, out, cache=cache, page_table=table, kv_len=i32(1, 1), prefix=prefix)
        assert kvc.read_result(att.res)[0] == kvc.ERR_TIMEOUT
        att.res.zero_()
        att.run(q, out, prefix=prefix)
        assert kvc.read_result(att.res)[0] == kvc.ERR_TIMEOUT
# the context is still usable: attention over the cache alone waits for no one
att.res.zero_()
att.run(q, out, cache=cache, page_table=table, kv_len=i32(1, 1))
assert kvc.read_result(att.res)[0] == kvc.OK
back = torch.zeros(2, 2, 2, 128, device="cuda")
kvc.cache_read(cache, table, i32(0, 0), i32(0, 1, 2), back)
want = back[1].transpose(0, 1).repeat_interleave(8, 1)  # one token each: its value row
assert (out.float() - want).abs().max() <= want.abs().max() * 2.0 ** -7
print("timeout-child: ok")
"""


def test_prefix_wait_timeout_reports_status():
    lib = os.path.join(ROOT, "transform_codec_b200", "libkvc_wait0.so")
    assert os.path.exists(lib), "the wait0 test build is missing (build.build_all())"
    env = dict(os.environ, KVC_BUILD_VARIANT="wait0")
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + CHILD], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "timeout-child: ok" in r.stdout


NAN_CHILD = r"""
import sys
import torch
sys.path.insert(0, ROOT)
import transform_codec_b200 as kvc
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
cache = kvc.QuantCache(kvc.CACHE_INT8, 2, 128, 16, 4)
k, v = (torch.randn(40, 2, 128, device="cuda").bfloat16() for _ in range(2))
kvc.cache_write(cache, k, v, torch.arange(40, device="cuda"))
good = dict(cache=cache, kv_len=i32(20, 20), page_table=i32(0, 1, 1, 2).reshape(2, 2))
bad = dict(good, page_table=i32(0, 77, 1, 2).reshape(2, 2))
for group in (8, 100):  # one tile of rows, and two
    q = torch.randn(2, 2 * group, 128, device="cuda").bfloat16()
    for tokens in (100, 2000):
        prefix = tuple(torch.randn(2, tokens, 128, device="cuda").bfloat16() for _ in range(2))
        att = kvc.Attention(torch.bfloat16, 2 * group, 2, 128, max_rows=2, max_seqs=2, max_kv=20, prefix_tokens=tokens)
        for kw, status in ((good, kvc.ERR_TIMEOUT), ({}, kvc.ERR_TIMEOUT), (bad, kvc.ERR_TIMEOUT)):
            out, lse = torch.zeros_like(q), torch.zeros(2, 2 * group, device="cuda")
            att.res.zero_()
            att.run(q, out, prefix=prefix, lse=lse, **kw)
            assert kvc.read_result(att.res)[0] == status, kvc.read_result(att.res)
            assert torch.isnan(out).all() and torch.isnan(lse).all()
            # a sequence that shares none of the prefix waits for nothing that its answer needs
            if kw is good:
                alone = torch.zeros_like(q)
                att.run(q, alone, **kw)
                att.run(q, out, prefix=prefix, prefix_len=i32(0, tokens), lse=lse, **kw)
                assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
                assert (out[0].float() - alone[0].float()).abs().max() <= 2.0 ** -7 * alone[0].float().abs().max()
print("nan-child: ok")
"""


def test_a_timeout_leaves_nan():
    """What a wait that gave up leaves behind is NaN, also after the join and where no result is asked for; a bad
    index in the same call does not hide the timeout."""
    env = dict(os.environ, KVC_BUILD_VARIANT="wait0")
    r = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\n" + NAN_CHILD], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "nan-child: ok" in r.stdout
