"""The serving cache's operators, as measured cases: writing tokens into a
quantised paged cache, reading token ranges back as slices, attention of a
batch's newest tokens over such a cache, and attention of a batch that shares a
long 16-bit prefix and continues in the cache.

A cache row is one (token, key/value, head): D codes and one fp32 scale s, value
= s * y with y the code's own value (E2M1: the 4-bit value times the e4m3 scale
of its block of 16 channels). Plain forms in fp32 torch operations; exact() in
fp64 from the definitions. Sizes are this repository's cache shapes (8 heads of
128 or 12 of 64, up to 32,768 tokens) with query groups of 1 to 16.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
PEAK = {"e4m3": 448.0, "int8": 127.0, "e2m1": 2688.0}  # largest |y| of a format
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one new token of one sequence: the launch is all there is
        dict(name="write one token", op="write", fmt="e4m3", dtype="bf16", tokens=1, heads=8, dim=128, page=64),
        # a padded step of a mixed batch, GPT-2-sized heads
        dict(name="write 1000 padded", op="write", fmt="int8", dtype="fp16", tokens=1000, heads=12, dim=64, page=16),
        # a decoded 32k-token layer put into 4-bit pages and checked by reading it back
        dict(name="write and read 32k", op="write", fmt="e2m1", dtype="bf16", tokens=32768, heads=8, dim=128, page=64),
        # one short sequence taken out of the cache
        dict(name="read 511", op="read", fmt="int8", dtype="fp16", batch=1, longest=511, heads=8, dim=128, page=16),
        # eight sequences exported as slices for the codec
        dict(name="read 8 ragged", op="read", fmt="e4m3", dtype="bf16", batch=8, longest=16384, heads=8, dim=128, page=64),
        # one user's next token, short context: latency
        dict(name="attend 1 x 1023", op="attend", fmt="e4m3", dtype="bf16", batch=1, longest=1023, queries=1,
             heads=8, group=8, dim=128, page=64, prefix=0),
        # one user's next token, long context: work split over the tokens
        dict(name="attend 1 x 131072", op="attend", fmt="int8", dtype="bf16", batch=1, longest=131072, queries=1,
             heads=8, group=8, dim=128, page=64, prefix=0),
        # a ragged batch on 4-bit pages
        dict(name="attend 64 ragged", op="attend", fmt="e2m1", dtype="fp16", batch=64, longest=8192, queries=1,
             heads=8, group=4, dim=128, page=32, prefix=0),
        # a full batch at 32k with drafted tokens to verify
        dict(name="attend 32 x 32768", op="attend", fmt="e4m3", dtype="bf16", batch=32, longest=32768, queries=4,
             heads=8, group=8, dim=128, page=64, prefix=0),
        # a short system prompt and a handful of sequences
        dict(name="shared 512 x 5", op="attend", fmt="int8", dtype="fp16", batch=5, longest=77, queries=1,
             heads=12, group=1, dim=64, page=16, prefix=512),
        # a long document and a small batch
        dict(name="shared 8192 x 16", op="attend", fmt="e2m1", dtype="fp16", batch=16, longest=300, queries=1,
             heads=8, group=8, dim=128, page=32, prefix=8192),
        # a long document and a large batch: products bound
        dict(name="shared 32768 x 128", op="attend", fmt="e4m3", dtype="bf16", batch=128, longest=500, queries=1,
             heads=8, group=8, dim=128, page=64, prefix=32768),
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "shared", "shared"])
    c = dict(op=op, fmt=rng.choice(["e4m3", "int8", "e2m1"]), dtype=rng.choice(["bf16", "fp16"]),
             heads=rng.choice([1, 2, 4, 5, 8, 12]), dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]))
    if op in ("write", "read"):
        c["dtype"] = rng.choice(["bf16", "fp16", "f32"])
        c["dim"] = rng.choice([32, 64, 96, 128, 256])
    if op == "write":
        c["tokens"] = _spread(rng, 1, 12000)
    elif op == "read":
        c.update(batch=rng.randint(1, 12), longest=_spread(rng, 1, 4000))
    else:
        c.update(op="attend", group=rng.choice([1, 2, 3, 4, 7, 8, 16]), queries=rng.choice([1, 1, 1, 2, 3, 5]))
        if op == "attend":
            batch = _spread(rng, 1, 100)
            c.update(batch=batch, longest=_spread(rng, 1, 600000 // max(batch, 8)), prefix=0)
        else:
            batch = _spread(rng, 1, 100)
            rows = c["heads"] * c["group"] * c["queries"] * batch  # no more products than the largest listed case
            c.update(batch=batch, longest=_spread(rng, 1, 600), prefix=_spread(rng, 1, min(20000, 8192 * 32768 // rows)))
    return c


# ---- lengths follow from the case alone

def _lengths(c):
    b, top = c["batch"], c["longest"]
    if b == 1:
        return [top]
    if c.get("queries", 1) > 1 and c["longest"] >= 16384:  # a full batch: nearly equal lengths
        return [top - 37 * i for i in range(b)]
    ls = [max(1, int(top * ((i * 0.6180339887) % 1.0))) for i in range(b)]
    ls[0] = top
    if b > 4:
        ls[3] = 0
    return ls


def _queries(c):
    return [1 + (i * 7) % c["queries"] for i in range(c["batch"])]


def _prefix_lengths(c):
    """Most of the batch shares all of the prefix; one sequence part of it, one nothing."""
    p = [c["prefix"]] * c["batch"]
    if c["batch"] > 2:
        p[1] = c["prefix"] // 3
    if c["batch"] > 4:
        p[4] = 0
    return p


def _pages(c):
    return [-(-n // c["page"]) for n in _lengths(c)]


def _row_bytes(c):
    return {"e4m3": c["dim"], "int8": c["dim"], "e2m1": c["dim"] // 2 + c["dim"] // 16}[c["fmt"]] + 4


def work(c):
    size, H, D = (4 if c["dtype"] == "f32" else 2), c["heads"], c["dim"]
    if c["op"] == "write":
        n = _written(c)
        b = n * 2 * H * (D * size + _row_bytes(c)) + 8 * c["tokens"]
        if c["fmt"] == "e2m1":
            b += n * 2 * H * (D * size + _row_bytes(c))
        return {"bytes": b, "flops": 4 * n * 2 * H * D}
    if c["op"] == "read":
        n = sum(_lengths(c))
        return {"bytes": n * 2 * H * (D * size + _row_bytes(c)), "flops": n * 2 * H * D}
    G = c["group"]
    lens, qs, pre = _lengths(c), _queries(c), _prefix_lengths(c)
    b = sum(lens) * 2 * H * _row_bytes(c) + 2 * c["prefix"] * H * D * size + sum(qs) * H * G * (2 * D * size + 4)
    f = sum(4 * n * H * G * D * (l + p) for l, n, p in zip(lens, qs, pre))
    return {"bytes": b, "flops": f}


# ---- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _written(c):
    """Tokens of a write that are not padding: every 13th is, from the sixth on."""
    return sum(1 for i in range(c["tokens"]) if i % 13 != 5)


def _empty_cache(c, pages, g):
    """A cache whose rows hold arbitrary earlier contents."""
    H, D, P = c["heads"], c["dim"], c["page"]
    width = D // 2 if c["fmt"] == "e2m1" else D
    codes = torch.randint(0, 120, (pages, 2, H, P, width), device="cuda", dtype=torch.uint8, generator=g)
    scales = torch.rand(pages, 2, H, P, device="cuda", generator=g)
    micro = None
    if c["fmt"] == "e2m1":
        micro = torch.randint(0, 120, (pages, 2, H, P, D // 16), device="cuda", dtype=torch.uint8, generator=g)
    return codes, scales, micro


def _full_cache(c, pages, g):
    """A cache as quantising writes leave it: codes up to the row's largest, scales of keys and values around one."""
    H, D, P = c["heads"], c["dim"], c["page"]
    if c["fmt"] == "int8":
        x = torch.randn(pages, 2, H, P, D, device="cuda", generator=g)
        codes = x.mul_(45.0).clamp_(-127, 127).to(torch.int8).view(torch.uint8)
    elif c["fmt"] == "e4m3":
        x = torch.randn(pages, 2, H, P, D, device="cuda", generator=g)
        codes = x.mul_(150.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes = torch.randint(0, 256, (pages, 2, H, P, D // 2), device="cuda", dtype=torch.uint8, generator=g)
    micro = None
    if c["fmt"] == "e2m1":
        u = torch.rand(pages, 2, H, P, D // 16, device="cuda", generator=g) * 300 + 148
        micro = u.to(torch.float8_e4m3fn).view(torch.uint8)
    std = {"int8": 45.0, "e4m3": 150.0, "e2m1": 900.0}[c["fmt"]]
    scales = torch.exp(torch.randn(pages, 2, H, P, device="cuda", generator=g) * 0.5) / std
    return codes, scales, micro


def _table(c, g):
    """Shuffled pages; entries past a sequence's last page are -1. Returns the table and the pages in the pool."""
    need = _pages(c)
    total = sum(need) + 3
    order = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    table = torch.full((c["batch"], max(max(need), 1) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _spoil(c, table, scales):
    """Rows behind each sequence's last token in its last page hold NaN scales."""
    P, lens = c["page"], _lengths(c)
    for b, n in enumerate(lens):
        if n % P:
            scales[table[b, n // P].long(), :, :, n % P:] = float("nan")


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _starts(v):
    s = [0]
    for x in v:
        s.append(s[-1] + x)
    return s


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    dt, H, D = DTYPES[c["dtype"]], c["heads"], c["dim"]
    s = {"case": c}
    if c["op"] == "write":
        N, P = c["tokens"], c["page"]
        # keys and values lie side by side, as a fused projection leaves them
        mean = torch.randn(1, 2 * H, D, device="cuda", generator=g)
        dev = torch.exp(0.5 * torch.randn(1, 2 * H, D, device="cuda", generator=g))
        kv = (mean + dev * torch.randn(N, 2 * H, D, device="cuda", generator=g)).to(dt)
        pages = -(-N // P) + 2
        slots = torch.randperm(pages * P - P, device="cuda", generator=g)[:N].clone()
        slots[5::13] = -1
        s.update(k=kv[:, :H], v=kv[:, H:], slots=slots)
        s["codes"], s["scales"], s["micro"] = _empty_cache(c, pages, g)
        if c["fmt"] == "e2m1":
            # read the same tokens back: one sequence whose pages are in the pool's order
            s["table"] = torch.arange(pages, device="cuda", dtype=torch.int32)[None]
            s["start"], s["out_start"] = _ints([0]), _ints([0, pages * P - P])
            s["out"] = torch.zeros(2, H, pages * P - P, D, dtype=dt, device="cuda")
    elif c["op"] == "read":
        lens = _lengths(c)
        s["table"], pages = _table(c, g)
        s["codes"], s["scales"], s["micro"] = _full_cache(c, pages, g)
        _spoil(c, s["table"], s["scales"])
        first = [n // 5 for n in lens]  # a part of each sequence, from an odd place on
        s["start"], s["out_start"] = _ints(first), _ints(_starts([n - f for n, f in zip(lens, first)]))
        s["total"] = sum(n - f for n, f in zip(lens, first))
        s["out"] = torch.zeros(2, H, s["total"] + 3, D, dtype=dt, device="cuda")
    else:
        G, qs = c["group"], _queries(c)
        n = sum(qs)
        s["table"], pages = _table(c, g)
        s["codes"], s["scales"], s["micro"] = _full_cache(c, pages, g)
        _spoil(c, s["table"], s["scales"])
        s["kv_len"] = _ints(_lengths(c))
        s["q_start"] = _ints(_starts(qs)) if c["queries"] > 1 else None
        s["q"] = (torch.randn(n, H * G, D, device="cuda", generator=g) * 1.5).to(dt)
        s["out"] = torch.zeros(n, H * G, D, dtype=dt, device="cuda")
        s["lse"] = torch.zeros(n, H * G, device="cuda")
        s["scale"] = D ** -0.5
        if c["prefix"]:
            s["pk"] = torch.randn(H, c["prefix"], D, device="cuda", generator=g).to(dt)
            s["pv"] = torch.randn(H, c["prefix"], D, device="cuda", generator=g).to(dt)
            s["prefix_len"] = _ints(_prefix_lengths(c))
    if own:  # the handles that a program keeps
        import transform_codec_b200 as kvc
        fmt = {"e4m3": kvc.CACHE_E4M3, "int8": kvc.CACHE_INT8, "e2m1": kvc.CACHE_E2M1}[c["fmt"]]
        s["cache"] = kvc.QuantCache(fmt, H, D, c["page"], s["codes"].shape[0], codes=s["codes"], scales=s["scales"],
                                    micro=s["micro"])
        if c["op"] == "attend":
            s["attention"] = kvc.Attention(s["q"].dtype, H * c["group"], H, D, max_rows=s["q"].shape[0],
                                           max_seqs=c["batch"], max_queries=c["queries"], max_kv=c["longest"],
                                           prefix_tokens=c["prefix"])
    return s


def run(s):
    c = s["case"]
    if c["op"] == "write":
        return _run_write(s, c)
    if c["op"] == "read":
        return _run_read(s, c)
    return _run_attend(s, c)


# ---- write

def _run_write(s, c):
    if own:
        import transform_codec_b200 as kvc
        kvc.cache_write(s["cache"], s["k"], s["v"], s["slots"])
        if c["fmt"] == "e2m1":
            kvc.cache_read(s["cache"], s["table"], s["start"], s["out_start"], s["out"])
    else:
        _plain_write(s, c)
        if c["fmt"] == "e2m1":
            _plain_read(s, c, s["out"].shape[2])
    if c["fmt"] == "e2m1":
        return {"values": s["out"], "scales": s["scales"], "micro": s["micro"].view(torch.float8_e4m3fn)}
    return {"codes": s["codes"].view(torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn), "scales": s["scales"]}


def _plain_write(s, c):
    x = torch.stack((s["k"], s["v"]), 1).float()  # [N][2][H][D]
    N, _, H, D = x.shape
    f32 = lambda v: torch.full((), v, dtype=torch.float32, device=x.device)  # noqa: E731
    top = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    scale = top * f32(1.0 / PEAK[c["fmt"]])
    scale = torch.where(top < 2.0 ** -96, torch.zeros_like(scale), scale)
    inv = torch.where(scale > 0, torch.ones_like(scale) / scale, torch.zeros_like(scale))
    live = (~bad) & (scale > 0)
    inv = torch.where(live, inv, torch.zeros_like(inv))
    x = torch.where(bad[..., None], torch.zeros_like(x), x)
    micro = None
    if c["fmt"] == "int8":
        codes = torch.round(x * inv[..., None]).clamp(-127, 127).to(torch.int8).view(torch.uint8)
    elif c["fmt"] == "e4m3":
        codes = (x * inv[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        blocks = x.reshape(N, 2, H, D // 16, 16)
        u = ((blocks.abs().amax(-1) * inv[..., None]) * f32(1.0 / 6.0)).clamp(max=448).to(torch.float8_e4m3fn)
        both = scale[..., None] * u.float()
        inv_b = torch.where(live[..., None] & (u.float() > 0), torch.ones_like(both) / both, torch.zeros_like(both))
        y = blocks * inv_b[..., None]
        a = y.abs()
        code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
        code = (code + 8 * torch.signbit(y)).to(torch.uint8).reshape(N, 2, H, D)
        codes = code[..., 0::2] | (code[..., 1::2] << 4)
        micro = u.view(torch.uint8)
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    page, at = slot // c["page"], slot % c["page"]
    s["codes"][page, :, :, at] = codes[keep]
    s["scales"][page, :, :, at] = scale[keep]
    if micro is not None:
        s["micro"][page, :, :, at] = micro[keep]


# ---- read

def _values(c, codes, scales, micro):
    """fp32 values of gathered rows: codes [...][width], scales [...], micro [...][D / 16]."""
    if c["fmt"] == "int8":
        y = codes.view(torch.int8).float()
    elif c["fmt"] == "e4m3":
        y = codes.view(torch.float8_e4m3fn).float()
    else:
        levels = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
        y = torch.stack((levels[(codes & 15).int()], levels[(codes >> 4).int()]), -1).flatten(-2)
        y = y * micro.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    return y * scales[..., None]


def _plain_read(s, c, total):
    n = s["out_start"][1:] - s["out_start"][:-1]
    seq = torch.repeat_interleave(torch.arange(n.shape[0], device=n.device), n.long(), output_size=total)
    pos = torch.arange(total, device=n.device) - s["out_start"][seq] + s["start"][seq]
    page, at = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    micro = s["micro"][page, :, :, at] if s["micro"] is not None else None
    x = _values(c, s["codes"][page, :, :, at], s["scales"][page, :, :, at], micro)  # [total][2][H][D]
    s["out"][:, :, :total] = x.permute(1, 2, 0, 3).to(s["out"].dtype)


def _run_read(s, c):
    if own:
        import transform_codec_b200 as kvc
        kvc.cache_read(s["cache"], s["table"], s["start"], s["out_start"], s["out"])
    else:
        _plain_read(s, c, s["total"])
    return s["out"]


# ---- attention

def _run_attend(s, c):
    if own:
        s["attention"].run(s["q"], s["out"], cache=s["cache"], page_table=s["table"], kv_len=s["kv_len"],
                           q_start=s["q_start"], prefix=(s["pk"], s["pv"]) if c["prefix"] else None,
                           prefix_len=s["prefix_len"] if c["prefix"] else None, lse=s["lse"], scale=s["scale"])
    else:
        _plain_attend(s, c)
    return {"out": s["out"], "lse": s["lse"]}


def _part(scores, values):
    """Largest score, sum of exponentials and weighted values over the last axis; rows with no score give zeros."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp(scores - top)
    return top, p.sum(-1, keepdim=True), p @ values


def _plain_attend(s, c):
    H, G, D, B, Q = c["heads"], c["group"], c["dim"], c["batch"], c["queries"]
    n = s["q"].shape[0]
    start = s["q_start"] if s["q_start"] is not None else torch.arange(n + 1, device="cuda", dtype=torch.int32)
    count = start[1:] - start[:-1]
    j = torch.arange(Q, device="cuda")
    rows = torch.minimum(start[:-1, None] + j, start[1:, None] - 1).long()  # [B][Q] query tokens
    # the sequence's own cache, padded to the longest
    table = s["table"].long().clamp(min=0)
    micro = s["micro"][table] if s["micro"] is not None else None
    kv = _values(c, s["codes"][table], s["scales"][table], micro)  # [B][pages][2][H][P][D]
    T = kv.shape[1] * kv.shape[4]
    t = torch.arange(T, device="cuda")
    there = t[None] < s["kv_len"][:, None]  # [B][T]
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, B, H, T, D)
    kv = torch.where(there[None, :, None, :, None], kv, torch.zeros((), device="cuda"))
    q = s["q"].float().reshape(n, H, G, D)
    qb = q[rows].permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    scores = (qb @ kv[0].transpose(-1, -2) * s["scale"]).reshape(B, H, Q, G, T)
    limit = s["kv_len"][:, None] - count[:, None] + j  # [B][Q]: the last token seen
    seen = t <= limit[..., None]
    scores = scores.masked_fill(~seen[:, None, :, None], float("-inf")).reshape(B, H, Q * G, T)
    top, total, acc = _part(scores, kv[1])
    del kv, scores
    pick = [x.reshape(B, H, Q, G, -1).permute(0, 2, 1, 3, 4) for x in (top, total, acc)]
    which = torch.searchsorted(start[1:].contiguous(), torch.arange(n, device="cuda", dtype=torch.int32), right=True)
    at = torch.arange(n, device="cuda") - start[which]
    top, total, acc = (x[which, at] for x in pick)  # [n][H][G][1 or D]
    if c["prefix"]:
        k, v = s["pk"].float(), s["pv"].float()
        qh = q.permute(1, 0, 2, 3).reshape(H, n * G, D)
        scores = qh @ k.transpose(-1, -2) * s["scale"]
        shared = torch.arange(c["prefix"], device="cuda")[None] < s["prefix_len"][which].repeat_interleave(G)[:, None]
        scores.masked_fill_(~shared, float("-inf"))
        part = [x.reshape(H, n, G, -1).permute(1, 0, 2, 3) for x in _part(scores, v)]
        none, both = total == 0, part[1] == 0
        high = torch.where(none, part[0], torch.where(both, top, torch.maximum(top, part[0])))
        a = torch.where(none, torch.zeros_like(top), torch.exp(top - high))
        b = torch.where(both, torch.zeros_like(top), torch.exp(part[0] - high))
        top, total, acc = high, total * a + part[1] * b, acc * a + part[2] * b
    out = torch.where(total > 0, acc / total, torch.zeros_like(acc))
    s["out"].copy_(out.reshape(n, H * G, D))
    s["lse"].copy_((top + torch.log(total)).reshape(n, H * G))


# ---- the definitions in 64 bits

def _exact_values(c, s, page, at):
    """fp64 values [rows][2][H][D] of the cache rows at (page, at)."""
    code = s["codes"][page, :, :, at]
    if c["fmt"] == "e2m1":
        nib = torch.stack((code & 15, code >> 4), -1).reshape(*code.shape[:-1], c["dim"]).long()
        e, m = (nib >> 1) & 3, nib & 1
        y = torch.where(e == 0, 0.5 * m.double(), (1 + 0.5 * m.double()) * torch.exp2((e - 1).double()))
        y = torch.where(nib >= 8, -y, y)
        u = s["micro"][page, :, :, at].view(torch.float8_e4m3fn).double()
        y = (y.reshape(*u.shape, 16) * u[..., None]).reshape(*code.shape[:-1], c["dim"])
    else:
        y = code.view(torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn).double()
    return y * s["scales"][page, :, :, at].double()[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "write":
        return _exact_write(s, c)
    if c["op"] == "read":
        out = s["out"].double()
        starts = s["out_start"].tolist()
        for b, first in enumerate(s["start"].tolist()):
            pos = torch.arange(first, first + starts[b + 1] - starts[b], device="cuda")
            x = _exact_values(c, s, s["table"][b].long()[pos // c["page"]], pos % c["page"])
            out[:, :, starts[b]:starts[b + 1]] = x.permute(1, 2, 0, 3)
        return out
    return _exact_attend(s, c)


def _exact_write(s, c):
    """Scales in 64 bits, and the value of each code nearest to x / s."""
    D, P = c["dim"], c["page"]
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    x = torch.stack((s["k"], s["v"]), 1)[keep].double()
    slot = s["slots"][keep]
    scale = x.abs().amax(-1) / PEAK[c["fmt"]]
    y = x / scale[..., None]
    page, at = slot // P, slot % P
    scales = s["scales"].double()
    scales[page, :, :, at] = scale
    if c["fmt"] == "int8":
        return {"codes": None, "scales": scales}  # whole numbers
    if c["fmt"] == "e4m3":
        codes = s["codes"].view(torch.float8_e4m3fn).double()
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        codes[page, :, :, at] = torch.round(y / step) * step
        return {"codes": codes, "scales": scales}
    b = y.reshape(*y.shape[:-1], D // 16, 16)
    u = b.abs().amax(-1) / 6
    step = torch.exp2(torch.floor(torch.log2(u.clamp(min=2.0 ** -6))) - 3)
    u = torch.round(u / step) * step
    r = torch.where(u[..., None] > 0, b / u[..., None], torch.zeros_like(b)).clamp(-6, 6)
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=1.0))) - 1)
    value = (torch.round(r / step) * step * u[..., None]).reshape(y.shape) * scale[..., None]
    micro = s["micro"].view(torch.float8_e4m3fn).double()
    micro[page, :, :, at] = u
    total = s["out"].shape[2]
    pos = torch.arange(total, device="cuda")
    out = _exact_values(c, s, pos // P, pos % P)
    out[slot] = value
    return {"values": out.permute(1, 2, 0, 3), "scales": scales, "micro": micro}


def _exact_attend(s, c):
    H, G, D, P = c["heads"], c["group"], c["dim"], c["page"]
    n = s["q"].shape[0]
    starts = s["q_start"].tolist() if s["q_start"] is not None else list(range(n + 1))
    lens = s["kv_len"].tolist()
    pre = s["prefix_len"].tolist() if c["prefix"] else [0] * c["batch"]
    out = torch.zeros(n, H, G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((n, H, G), float("-inf"), dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        pos = torch.arange(lens[b], device="cuda")
        kv = _exact_values(c, s, s["table"][b].long()[pos // P], pos % P).permute(1, 2, 0, 3)  # [2][H][T][D]
        k, v = kv[0], kv[1]
        if pre[b]:
            k = torch.cat((s["pk"][:, :pre[b]].double(), k), 1)
            v = torch.cat((s["pv"][:, :pre[b]].double(), v), 1)
        first, last = starts[b], starts[b + 1]
        m = last - first
        q = s["q"][first:last].double().reshape(m, H, G, D).permute(1, 0, 2, 3).reshape(H, m * G, D)
        z = (q @ k.transpose(1, 2)).reshape(H, m, G, -1) * s["scale"]
        for i in range(m):
            sees = pre[b] + max(0, lens[b] - m + i + 1)
            if sees <= 0:
                continue
            l = torch.logsumexp(z[:, i, :, :sees], -1)
            lse[first + i] = l
            out[first + i] = torch.exp(z[:, i, :, :sees] - l[..., None]) @ v[:, :sees]
    return {"out": out.reshape(n, H * G, D), "lse": lse.reshape(n, H * G)}
