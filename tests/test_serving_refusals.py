"""The serving cache's entry points refuse bad arguments before any launch (CPU
only): a child process that sees no CUDA device calls the C ABI with device
addresses that are never dereferenced."""
import ctypes
import json
import os
import subprocess
import sys

import pytest
import torch

import transform_codec_b200 as kvc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import ctypes, json
import transform_codec_b200 as kvc

lib = kvc._lib
A = 0x7F0000000000
vp, ref = ctypes.c_void_p, ctypes.byref
out = {}

def cache(**kw):
    d = dict(format=kvc.CACHE_E2M1, n_heads=2, head_dim=64, page_tokens=16, n_pages=4, reserved=0, codes=A, scales=A,
             micro=A)
    d.update(kw)
    return kvc.CacheDesc(**d)

def write(name, c=None, dtype=kvc.BF16, n=3, k=A, kt=128, kh=64, v=A, vt=128, vh=64, slots=A, res=A):
    c = cache() if c is None else c
    out["write " + name] = lib.kvc_cache_write(ref(c), dtype, n, k, kt, kh, v, vt, vh, slots, res, None)

def read(name, c=None, dtype=kvc.BF16, seqs=2, pages=A, stride=4, start=A, out_start=A, dst=A, tokens=5, res=A):
    c = cache() if c is None else c
    out["read " + name] = lib.kvc_cache_read(ref(c), dtype, seqs, pages, stride, start, out_start, dst, tokens, res,
                                             None)

def attend(name, ws=A, ws_bytes=1 << 30, res=A, c=None, **kw):
    c = cache() if c is None else c
    d = dict(dtype=kvc.BF16, n_rows=4, n_q_heads=8, n_heads=2, head_dim=64, n_seqs=4, max_queries=1, max_kv=5000,
             scale=1.0, prefix_tokens=300, q=A, q_token_stride=512, q_head_stride=64, out=A, out_token_stride=512,
             out_head_stride=64, lse=A, q_start=A, cache=ctypes.pointer(c), pages=A, kv_len=A, pages_stride=4,
             reserved=0, prefix_k=A, prefix_v=A, prefix_head_stride=300 * 64, prefix_len=A)
    d.update(kw)
    desc = kvc.AttendDesc(**d)
    out["attend " + name] = lib.kvc_attend(ref(desc), ws, ws_bytes, res, None)
    out["min " + name] = lib.kvc_attend_workspace_min(ref(desc))
    out["best " + name] = lib.kvc_attend_workspace_bytes(ref(desc))

for name, bad in (("format 0", dict(format=0)), ("format 4", dict(format=4)), ("no heads", dict(n_heads=0)),
                  ("head_dim 48", dict(head_dim=48)), ("head_dim 288", dict(head_dim=288)),
                  ("head_dim 0", dict(head_dim=0)), ("page 24", dict(page_tokens=24)),
                  ("page 8", dict(page_tokens=8)), ("page 2048", dict(page_tokens=2048)),
                  ("no pages", dict(n_pages=0)), ("reserved", dict(reserved=1)), ("no codes", dict(codes=None)),
                  ("no scales", dict(scales=None)), ("no micro", dict(micro=None)),
                  ("micro of int8", dict(format=kvc.CACHE_INT8)), ("codes misaligned", dict(codes=A + 8)),
                  ("scales misaligned", dict(scales=A + 4)), ("micro misaligned", dict(micro=A + 2))):
    write(name, cache(**bad))
    read(name, cache(**bad))
    attend(name, c=cache(**bad))
write("dtype", dtype=4)
write("no k", k=None)
write("no v", v=None)
write("no slots", slots=None)
write("k misaligned", k=A + 2)
write("slots misaligned", slots=A + 4)
write("res misaligned", res=A + 4)
write("token stride", kt=129)
write("head stride", vh=68)
write("f32 stride", dtype=kvc.F32, kt=130)
read("dtype", dtype=0)
read("no pages", pages=None)
read("no stride", stride=0)
read("no start", start=None)
read("no out_start", out_start=None)
read("no out", dst=None)
read("out misaligned", dst=A + 8)
read("start misaligned", start=A + 2)
attend("f32", dtype=kvc.F32)
attend("query heads", n_q_heads=7)
attend("no heads", n_heads=0)
attend("cache heads", n_heads=4)
attend("cache head_dim", head_dim=128)
attend("nothing to see", cache=None, prefix_tokens=0)
attend("scale", scale=float("nan"))
attend("no q", q=None)
attend("q misaligned", q=A + 8)
attend("out misaligned", out=A + 8)
attend("q stride", q_token_stride=516)
attend("out stride", out_head_stride=68)
attend("no pages", pages=None)
attend("no lengths", kv_len=None)
attend("no page stride", pages_stride=0)
attend("rows without starts", q_start=None, n_seqs=5)
attend("no prefix keys", prefix_k=None)
attend("prefix misaligned", prefix_v=A + 8)
attend("prefix stride", prefix_head_stride=300 * 64 + 4)
attend("prefix heads overlap", prefix_head_stride=299 * 64)
attend("prefix stride negative", prefix_head_stride=-300 * 64)
attend("reserved", reserved=1)
attend("lse misaligned", lse=A + 2)
attend("lengths misaligned", kv_len=A + 2)
attend("ws misaligned", ws=A + 8)
attend("too many rows", n_rows=1 << 30)
attend("too many sequences", n_seqs=1 << 17)
print(json.dumps(out))
'''
UNSUPPORTED = r'''
attend("head_dim 96", head_dim=96, c=cache(head_dim=96))
attend("head_dim 256", head_dim=256, c=cache(head_dim=256))
'''
FINE = r'''
write("nothing", n=0, k=None, v=None, slots=None)
read("no sequences", seqs=0, pages=None, start=None)
read("no tokens", tokens=0, dst=None)
attend("no rows", n_rows=0, n_seqs=0)
'''


def _child(code):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
    return json.loads(p.stdout.strip().splitlines()[-1])


def _calls(part):
    """The definitions, followed by these calls alone."""
    head = CHILD[:CHILD.index("for name, bad in")]
    return _child(head + part + "\nprint(json.dumps(out))\n")


def test_bad_arguments_are_refused():
    got = _child(CHILD)
    calls = {k: v for k, v in got.items() if not k.startswith(("min ", "best "))}
    assert len(calls) > 90
    wrong = {k: v for k, v in calls.items() if v != kvc.ERR_INVALID}
    assert not wrong, wrong


def test_unsupported_head_dims():
    got = _calls(UNSUPPORTED)
    assert {v for k, v in got.items() if k.startswith("attend")} == {kvc.ERR_UNSUPPORTED}
    assert {v for k, v in got.items() if k.startswith(("min", "best"))} == {0}


CAPACITY = r'''
attend("no workspace", ws=None, ws_bytes=0)
attend("one byte short", ws_bytes=2 * 4 * 8 * 4 * (64 + 1) - 1)   # two parts of every row: o and L
'''


def test_workspace_below_the_least():
    got = _calls(CAPACITY)
    assert {v for k, v in got.items() if k.startswith("attend")} == {kvc.ERR_CAPACITY}
    assert {v for k, v in got.items() if k.startswith("min")} == {2 * 4 * 8 * 4 * (64 + 1)}
    assert all(v > 2 * 4 * 8 * 4 * (64 + 1) for k, v in got.items() if k.startswith("best"))


def test_empty_calls_launch_nothing():
    got = _calls(FINE)
    assert {v for k, v in got.items() if not k.startswith(("min", "best"))} == {kvc.OK}


def test_cache_bytes():
    sizes = [ctypes.c_size_t() for _ in range(3)]
    refs = [ctypes.byref(s) for s in sizes]
    d = kvc.CacheDesc(kvc.CACHE_E2M1, 8, 128, 64, 1 << 20, 0, None, None, None)
    assert kvc.lib().kvc_cache_bytes(ctypes.byref(d), *refs) == kvc.OK
    rows = (1 << 20) * 2 * 8 * 64
    assert [s.value for s in sizes] == [rows * 64, rows * 4, rows * 8]
    d.format = kvc.CACHE_INT8
    assert kvc.lib().kvc_cache_bytes(ctypes.byref(d), *refs) == kvc.OK
    assert [s.value for s in sizes] == [rows * 128, rows * 4, 0]
    assert kvc.lib().kvc_cache_bytes(ctypes.byref(d), None, None, None) == kvc.OK
    assert kvc.lib().kvc_cache_bytes(None, *refs) == kvc.ERR_INVALID


@pytest.mark.parametrize("args", [(9, 2, 64, 16, 4), (kvc.CACHE_INT8, 0, 64, 16, 4), (kvc.CACHE_INT8, 2, 60, 16, 4),
                                  (kvc.CACHE_INT8, 2, 64, 20, 4), (kvc.CACHE_INT8, 2, 64, 16, 0),
                                  (kvc.CACHE_INT8, 2, 64, 16, 1 << 31), (kvc.CACHE_INT8, -1, 64, 16, 4)])
def test_binding_refuses_cache_shapes(args):
    with pytest.raises(kvc.KvcError) as e:
        kvc.QuantCache(*args, device="cpu")
    assert e.value.status == kvc.ERR_INVALID


def test_binding_refuses_tensors():
    """Shapes, types, strides and devices, before the library is called."""
    c = kvc.QuantCache(kvc.CACHE_E2M1, 2, 64, 16, 4, device="cpu")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    i = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    out = torch.zeros(2, 2, 5, 64, dtype=torch.bfloat16)
    bad = [lambda: kvc.cache_write(c, k[:2], k, slots), lambda: kvc.cache_write(c, k, k.float(), slots),
           lambda: kvc.cache_write(c, k, k, slots.int()), lambda: kvc.cache_write(c, k[:, :1], k[:, :1], slots),
           lambda: kvc.cache_write(c, k.transpose(1, 2).contiguous().transpose(1, 2), k, slots),
           lambda: kvc.cache_write(c, k.to("meta"), k, slots), lambda: kvc.cache_write(c, k, k, slots[:, None]),
           lambda: kvc.cache_write(c, k, k, slots[0]), lambda: kvc.cache_write(c, k, k, slots),  # tensors on the CPU
           lambda: kvc.cache_read(c, i(0, 1)[None], i(0)[0], i(0, 5), out),
           lambda: kvc.cache_read(c, i(0, 1)[None], i(0), i(0, 5), out),
           lambda: kvc.cache_read(c, i(0, 1)[None], i(0), i(0, 5), out.double()),
           lambda: kvc.cache_read(c, i(0, 1), i(0), i(0, 5), out),
           lambda: kvc.cache_read(c, i(0, 1)[None], i(0), i(0, 5, 6), out),
           lambda: kvc.cache_read(c, i(0, 1)[None].long(), i(0), i(0, 5), out),
           lambda: kvc.cache_read(c, i(0, 1)[None], i(0), i(0, 5), out[:, :1]),
           lambda: kvc.cache_read(c, i(0, 1)[None], i(0), i(0, 5), out.transpose(0, 1)),
           lambda: kvc.QuantCache(kvc.CACHE_INT8, 2, 64, 16, 4, codes=torch.zeros(4, 2, 2, 16, 32, dtype=torch.uint8)),
           lambda: kvc.QuantCache(kvc.CACHE_INT8, 2, 64, 16, 4, device="cpu", micro=c.micro),
           lambda: kvc.Attention(torch.float32, 8, 2, 64, 4, 4, device="cpu"),
           lambda: kvc.Attention(torch.int32, 8, 2, 64, 4, 4, device="cpu"),
           lambda: kvc.Attention(torch.bfloat16, 7, 2, 64, 4, 4, device="cpu")]
    for n, f in enumerate(bad):
        with pytest.raises(kvc.KvcError) as e:
            f()
        assert e.value.status == kvc.ERR_INVALID, n
    with pytest.raises(kvc.KvcError) as e:
        kvc.Attention(torch.bfloat16, 8, 2, 96, 4, 4, device="cpu")
    assert e.value.status == kvc.ERR_UNSUPPORTED
    a = kvc.Attention(torch.bfloat16, 8, 2, 64, 4, 4, max_kv=60, prefix_tokens=9, device="cpu")
    q, o = torch.zeros(4, 8, 64, dtype=torch.bfloat16), torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(4, 4, dtype=torch.int32), i(1, 2, 3, 4)
    p = torch.zeros(2, 9, 64, dtype=torch.bfloat16)
    runs = [dict(q=q[0], out=o[0]), dict(), dict(q=q.half()), dict(out=o[:3]), dict(q=q[:, :4], out=o[:, :4]),
            dict(kv_len=i(1, 2)),
            dict(kv_len=lens.long()), dict(page_table=table[:2]), dict(page_table=None), dict(q_start=i(0, 1, 2)),
            dict(prefix=(p, p[:, :5])), dict(prefix=(p.transpose(1, 2), p.transpose(1, 2))),
            dict(prefix=(p[:1], p[:1])), dict(prefix_len=i(1)), dict(lse=torch.zeros(4, 4)),
            dict(lse=torch.zeros(4, 8).half()), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))]
    for n, r in enumerate(runs):
        kw = dict(q=q, out=o, cache=c, page_table=table, kv_len=lens)
        kw.update(r)
        with pytest.raises(kvc.KvcError) as e:
            a.run(kw.pop("q"), kw.pop("out"), **kw)
        assert e.value.status == kvc.ERR_INVALID, n


@pytest.mark.parametrize("change", [
    dict(max_rows=70000, max_seqs=70000), dict(max_rows=-1), dict(max_rows=1 << 26, n_q_heads=64), dict(max_seqs=-1),
    dict(max_seqs=1 << 16), dict(max_queries=-1), dict(max_queries=1 << 32), dict(max_kv=1 << 31), dict(max_kv=-5),
    dict(prefix_tokens=1 << 31), dict(prefix_tokens=-1), dict(n_heads=0), dict(n_heads=-2), dict(n_q_heads=1 << 17),
    dict(n_q_heads=0), dict(max_rows=4.0), dict(max_kv=None),
])
def test_binding_refuses_attention_sizes(change):
    """A size that no call accepts is refused where it is given, not by the first call."""
    kw = dict(n_q_heads=8, n_heads=2, head_dim=64, max_rows=4, max_seqs=4)
    with pytest.raises(kvc.KvcError) as e:
        kvc.Attention(torch.bfloat16, device="cpu", **{**kw, **change})
    assert e.value.status == kvc.ERR_INVALID


def test_binding_accepts_the_largest_attention_sizes():
    a = kvc.Attention(torch.bfloat16, 8, 2, 64, max_rows=65535, max_seqs=65535, max_kv=1, device="cpu")
    assert a.workspace.numel() >= 16
    assert kvc.lib().kvc_attend_workspace_min(a._ref) == 0  # one part a row


@pytest.mark.parametrize("res", [lambda: torch.zeros(2, dtype=torch.int64, device="meta"),
                                 lambda: torch.zeros(1, dtype=torch.int64), lambda: torch.zeros(3, dtype=torch.int32),
                                 lambda: torch.zeros(4, dtype=torch.int64)[::2]])
def test_binding_refuses_results(monkeypatch, res):
    """A result on another device, or without room for a kvc_result, never reaches the library."""
    def launched(*args):
        raise AssertionError("launched")
    monkeypatch.setattr(kvc, "_launch", launched)
    c = kvc.QuantCache(kvc.CACHE_INT8, 2, 64, 16, 4, device="cpu")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    a = kvc.Attention(torch.bfloat16, 8, 2, 64, 4, 4, max_kv=60, device="cpu")
    q = torch.zeros(1, 8, 64, dtype=torch.bfloat16)
    calls = [lambda r: kvc.cache_write(c, k, k, torch.zeros(3, dtype=torch.int64), res=r),
             lambda r: kvc.cache_read(c, i(0)[None], i(0), i(0, 5), torch.zeros(2, 2, 5, 64), res=r),
             lambda r: a.run(q, q.clone(), cache=c, page_table=i(0)[None], kv_len=i(1), res=r)]
    for call in calls:
        with pytest.raises(kvc.KvcError) as e:
            call(res())
        assert e.value.status == kvc.ERR_INVALID
        with pytest.raises(AssertionError):  # a good one does
            call(torch.zeros(2, dtype=torch.int64))


EMPTY = r'''
none = dict(q=None, out=None, lse=None, pages=None, kv_len=None, prefix_k=None, prefix_v=None, prefix_len=None)
attend("no rows", n_rows=0, n_seqs=0, q_start=None, c=cache(codes=None, scales=None, micro=None), **none)
attend("no sequences", n_seqs=0, **dict(none, q=A, out=A, lse=A))
attend("sequences without rows", n_rows=0, **none)
attend("no prefix", n_rows=0, n_seqs=0, prefix_tokens=0, ws=None, ws_bytes=0, **none)
'''
EMPTY_BAD = r'''
attend("shape", n_rows=0, n_seqs=0, n_q_heads=7)
attend("cache shape", n_rows=0, n_seqs=0, c=cache(page_tokens=24))
attend("a sequence without a row", n_rows=0, n_seqs=1, q_start=None)
attend("nothing to see", n_rows=0, n_seqs=0, cache=None, prefix_tokens=0)
'''


def test_empty_attention_needs_no_arrays():
    """Empty tensors have no address; shapes are looked at all the same."""
    got = _calls(EMPTY)
    assert {v for k, v in got.items() if k.startswith("attend")} == {kvc.OK}, got
    got = _calls(EMPTY_BAD)
    assert {v for k, v in got.items() if k.startswith("attend")} == {kvc.ERR_INVALID}, got


def _workspace(**kw):
    d = dict(n_q_heads=64, n_heads=8, head_dim=128, max_rows=1, max_seqs=1, device="cpu")
    return kvc.Attention(torch.bfloat16, **{**d, **kw}).workspace.numel()


def test_a_length_that_is_not_known_is_split_like_a_long_one():
    """One query of 64 heads: the same parts as for 131,072 tokens. The workspace is bounded, and a prefix keeps its
    own parts."""
    assert _workspace() == _workspace(max_kv=131072) > 64 * 64 * 129 * 4
    assert _workspace(max_kv=1) == 16
    for rows, seqs in ((64, 1), (64, 64), (4096, 1), (65535, 65535)):
        prefix = _workspace(max_rows=rows, max_seqs=seqs, prefix_tokens=8192, max_kv=1)
        both = _workspace(max_rows=rows, max_seqs=seqs, prefix_tokens=8192)
        one = rows * 64 * 129 * 4
        assert prefix <= both <= prefix + max(32 << 20, one)
