"""Plain statements of the serving cache's operators for the tests: the
quantiser in the fp32 steps that define the codes, values and attention in
fp64, and the error that attention's roundings may cause."""
import math

import numpy as np
import torch

import transform_codec_b200 as kvc

FORMATS = {"e4m3": kvc.CACHE_E4M3, "int8": kvc.CACHE_INT8, "e2m1": kvc.CACHE_E2M1}
PEAK = {kvc.CACHE_E4M3: 448.0, kvc.CACHE_INT8: 127.0, kvc.CACHE_E2M1: 2688.0}
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float32)


def quantise(fmt, x):
    """codes uint8 [..., row bytes], scales fp32 [...], micro uint8 [..., D / 16] or None of x [..., D] (CPU)."""
    x = x.float()
    bad = ~torch.isfinite(x).all(-1)
    x = torch.where(bad[..., None], torch.zeros(()), x)
    top = x.abs().amax(-1)
    one = torch.ones(())
    scale = torch.where(top >= 2.0 ** -96, top * torch.tensor(np.float32(1.0) / np.float32(PEAK[fmt])), torch.zeros(()))
    inv = torch.where(scale > 0, one / scale, torch.zeros(()))
    micro = None
    if fmt == kvc.CACHE_INT8:
        codes = torch.round(x * inv[..., None]).clamp(-127, 127).to(torch.int8).view(torch.uint8)
    elif fmt == kvc.CACHE_E4M3:
        codes = (x * inv[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        b = x.reshape(*x.shape[:-1], -1, 16)
        sixth = torch.tensor(np.float32(1.0) / np.float32(6.0))
        u = ((b.abs().amax(-1) * inv[..., None]) * sixth).clamp(max=448).to(torch.float8_e4m3fn)
        both = scale[..., None] * u.float()
        y = b * torch.where(u.float() > 0, one / both, torch.zeros(()))[..., None]
        a = y.abs().numpy()
        # nearest level, ties to the even one: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
        code = sum(((a > t) if up else (a >= t)).astype(np.uint8) for t, up in
                   ((0.25, 1), (0.75, 0), (1.25, 1), (1.75, 0), (2.5, 1), (3.5, 0), (5.0, 1)))
        code = torch.from_numpy(code + 8 * np.signbit(y.numpy()).astype(np.uint8)).reshape(x.shape)
        codes = code[..., 0::2] | (code[..., 1::2] << 4)
        micro = u.view(torch.uint8)
    return codes, torch.where(bad, torch.tensor(float("nan")), scale), micro


def code_values(fmt, codes, micro):
    """fp64 y of codes."""
    if fmt == kvc.CACHE_INT8:
        return codes.view(torch.int8).double()
    if fmt == kvc.CACHE_E4M3:
        return codes.view(torch.float8_e4m3fn).double()
    lv = torch.from_numpy(np.concatenate([LEVELS, -LEVELS]).astype(np.float64))
    y = torch.stack((lv[(codes & 15).long()], lv[(codes >> 4).long()]), -1).flatten(-2)
    return y * micro.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def signless(fmt, codes):
    """Codes with the sign of zeros cleared: -0 and 0 stand for the same value."""
    c = codes.clone()
    if fmt == kvc.CACHE_E4M3:
        return torch.where(c == 0x80, torch.zeros_like(c), c)
    if fmt == kvc.CACHE_E2M1:
        c = torch.where((c & 15) == 8, c & 0xF0, c)
        return torch.where((c >> 4) == 8, c & 0x0F, c)
    return c


class HostCache:
    """A cache on the CPU and the same on the GPU, filled at random; pages of the
    sequences are shuffled, everything behind their ends holds NaN scales."""

    def __init__(self, fmt, heads, dim, page, lens, seed=0, spread=1.0, extra_pages=2):
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.fmt, self.heads, self.dim, self.page, self.lens = fmt, heads, dim, page, list(lens)
        n_pages = sum(need) + extra_pages
        x = torch.from_numpy(rng.standard_normal((n_pages, 2, heads, page, dim)).astype(np.float32))
        x *= torch.from_numpy(np.exp(spread * rng.standard_normal((n_pages, 2, heads, page, 1))).astype(np.float32))
        self.codes, self.scales, self.micro = quantise(fmt, x)
        order = rng.permutation(n_pages)
        self.table = torch.full((len(lens), max(max(need, default=1), 1) + 1), -1, dtype=torch.int32)
        used = torch.zeros(n_pages, page, dtype=torch.bool)
        at = 0
        for b, n in enumerate(need):
            ids = order[at:at + n]
            at += n
            self.table[b, :n] = torch.from_numpy(ids.astype(np.int32))
            for p, i in enumerate(ids):
                used[i, :max(0, min(page, lens[b] - p * page))] = True
        self.scales[~used[:, None, None].expand_as(self.scales)] = float("nan")
        if fmt == kvc.CACHE_E4M3:  # NaN codes too
            self.codes[~used[:, None, None].expand(n_pages, 2, heads, page)] = 0x7F
        if self.micro is not None:
            self.micro[~used[:, None, None].expand(n_pages, 2, heads, page)] = 0x7F

    def gpu(self):
        return kvc.QuantCache(self.fmt, self.heads, self.dim, self.page, self.codes.shape[0], codes=self.codes.cuda(),
                              scales=self.scales.cuda(), micro=None if self.micro is None else self.micro.cuda())

    def values(self, b, parts=False):
        """fp64 [2][heads][n][dim] of sequence b's tokens; parts: code values and scales [2][heads][n] instead."""
        pos = torch.arange(self.lens[b])
        page = self.table[b].long()[pos // self.page]
        at = pos % self.page
        micro = None if self.micro is None else self.micro[page, :, :, at]
        y = code_values(self.fmt, self.codes[page, :, :, at], micro)
        scale = self.scales[page, :, :, at].double()
        if parts:
            return y.permute(1, 2, 0, 3), scale.permute(1, 2, 0)
        return (y * scale[..., None]).permute(1, 2, 0, 3)


def attention(q, starts, host=None, prefix=None, prefix_len=None, scale=1.0):
    """fp64 attention and the bound of each output's error before it is rounded
    to its type, for q [n][Hq][D] (CPU, 16-bit): out, lse and (bounds of out, bounds of lse).

    Roundings: weights enter the second product in 16 bits, off by at most u_p =
    2^-8 (bf16) or 2^-11 (fp16) of themselves, or by half of fp16's smallest step,
    2^-25, where the largest weight is 2^7 or more (a weight of a cache token
    holds its value scale; the codes are the other factor); scores are fp32 sums of D products, each
    partial sum off by 2^-23 of the sum of magnitudes at most (truncating adders
    included), which moves a weight by that much relative to itself, twice
    (itself and the sum); q as fp16 next to its largest element of 2^7 or more
    loses 2^-25 at most of each, under one such step; exp2, logarithms of scales
    and the joins add a few fp32 steps, counted as 2^-18."""
    n, Hq, D = q.shape
    H = host.heads if host is not None else prefix[0].shape[0]
    G = Hq // H
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64)
    tol = torch.zeros(n, Hq, D, dtype=torch.float64)
    ltol = torch.zeros(n, Hq, dtype=torch.float64)
    u_p = torch.finfo(q.dtype).eps / 2
    for b in range(len(starts) - 1):
        first, last = starts[b], starts[b + 1]
        m = last - first
        kv = host.values(b) if host is not None else torch.zeros(2, H, 0, D, dtype=torch.float64)
        p = 0 if prefix is None else (prefix[0].shape[1] if prefix_len is None else int(prefix_len[b]))
        k, v = kv[0], kv[1]
        if p:
            k = torch.cat((prefix[0][:, :p].double(), k), 1)
            v = torch.cat((prefix[1][:, :p].double(), v), 1)
        own = kv.shape[2]
        if own:
            codes, scales = host.values(b, parts=True)
            y, sv = codes[1], scales[1]
        for i in range(m):
            sees = p + max(0, own - m + i + 1)
            if not sees:
                continue
            x = q[first + i].double().reshape(H, G, D)
            z = torch.einsum("hgd,htd->hgt", x, k[:, :sees]) * scale
            mag = torch.einsum("hgd,htd->hgt", x.abs(), k[:, :sees].abs()) * abs(scale)
            l = torch.logsumexp(z, -1)
            w = torch.exp(z - l[..., None])
            lse[first + i] = l.reshape(Hq)
            out[first + i] = (w @ v[:, :sees]).reshape(Hq, D)
            weight = w @ v[:, :sees].abs()
            step = 2.0 ** -23 * (D + 8) * mag.amax(-1, keepdim=True)
            low = 2.0 ** -32 * w[..., :p].amax(-1, keepdim=True) * v[:, :p].abs().sum(1)[:, None] if p else 0.0
            if sees > p:
                biggest = (w[..., p:] * sv[:, None, :sees - p]).amax(-1, keepdim=True)
                low = low + 2.0 ** -32 * biggest * y[:, :sees - p].abs().sum(1)[:, None]
            ltol[first + i] = (step + 2.0 ** -18 + 2.0 ** -23 * l.abs()[..., None]).reshape(Hq)
            tol[first + i] = ((u_p + 2 * step + 2.0 ** -18) * weight + low).reshape(Hq, D)
    return out, lse, (tol, ltol)


def check_out(got, lse_got, want, lse, tol):
    """got within tol[0] plus its own rounding (half a step, or half the smallest one) of want; lse within tol[1]."""
    tol, ltol = tol
    f = torch.finfo(got.dtype)
    g = got.double().cpu()
    bound = tol + (want.abs() + tol) * (f.eps / 2) + f.smallest_normal * f.eps / 2
    off = (g - want).abs()
    assert torch.isfinite(g).all()
    worst = (off / bound).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"off by {worst} of the bound"
    if lse_got is not None:
        lg = lse_got.double().cpu()
        none = torch.isinf(lse)
        assert torch.equal(torch.isinf(lg), none)
        assert ((lg - lse).abs() <= ltol)[~none].all()
