"""Plain 64-bit forms of the 4-bit paged cache operators, and batches to test them on
(host-side; shared by the GPU tests)."""
import math

import torch

from paged_ref import TYPES, U, rotate

GROUP = 64
BITS = {torch.bfloat16: 4, torch.float16: 7}          # significant bits of a scale
LEAST = {torch.bfloat16: 2.0 ** -129, torch.float16: 2.0 ** -20}   # its smallest step


def quantize(x):
    """Codes (uint8, one each), scales and zeros (fp64, one per 64) of 16-bit values [..., D]."""
    dt = x.dtype
    g = x.double().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
    want = (hi - lo) / torch.full_like(hi, 15.0)
    m, e = torch.frexp(want)
    # (torch.ldexp multiplies by a power of two computed in 32 bits, on the GPU not exactly)
    s = torch.ceil(m * 2.0 ** BITS[dt]) * ((e.long() - BITS[dt] + 1023) << 52).view(torch.float64)
    s = torch.maximum(s, torch.ceil(want / LEAST[dt]) * LEAST[dt])
    d = torch.where(s > 0, s, torch.ones_like(s))
    z = torch.round(-lo / d).clamp(0, 15)
    c = (torch.round(g / d[..., None]) + z[..., None]).clamp(0, 15)
    v, most = (c - z[..., None]) * s[..., None], torch.finfo(dt).max
    c = c - (v > most).double() + (v < -most).double()
    return c.flatten(-2).to(torch.uint8), s, z


def patterns(s, z, dt):
    """Scale patterns [..., D / 64] of type dt."""
    return ((s.to(dt).view(torch.int16) & -16) | z.to(torch.int16)).view(dt)


def pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def unpack(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def values(codes, pats):
    """fp64 values of packed codes [..., D / 2] with their patterns [..., D / 64]."""
    bits = pats.contiguous().view(torch.int16)
    s, z = (bits & -16).view(pats.dtype).double(), (bits & 15).double()
    return ((unpack(codes).double().unflatten(-1, (-1, GROUP)) - z[..., None]) * s[..., None]).flatten(-2)


def empty_cache(pages, page, hk, D, dt, layout, device):
    """A pool whose every slot reads back as NaN."""
    def pool(last, dtype, fill):
        if layout == "hnd":
            return torch.full((pages, hk, page, last), fill, device=device, dtype=dtype).permute(0, 2, 1, 3)
        if layout == "nhd":
            return torch.full((pages, page, hk, last), fill, device=device, dtype=dtype)
        # rows with room between them
        return torch.full((pages, page, hk, 2 * last + 16), fill, device=device, dtype=dtype)[..., 16:16 + last]
    k, v = pool(D // 2, torch.uint8, 0xa7), pool(D // 2, torch.uint8, 0x3c)
    s = pool(D // 32, torch.int16, 0x7ff0)
    return k, v, s.view(dt)


class Batch4:
    """A 4-bit cache and a batch of sequences with `ql` new tokens and `kl` keys (the new
    ones included).  Slots that belong to no key read back as NaN."""

    def __init__(self, ql, kl, q_heads, kv_heads, D, dtype="bf16", page=16, layout="hnd", seed=0, device="cuda",
                 spread=1.0, extra_blocks=0, fill=True):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        dt = TYPES[dtype]
        self.ql, self.kl, self.hq, self.hk, self.D, self.page, self.dt = ql, kl, q_heads, kv_heads, D, page, dt
        B = len(ql)
        used = [-(-n // page) for n in kl]
        blocks = max(used + [1]) + extra_blocks
        pages = sum(used) + 2
        self.k_cache, self.v_cache, self.scales = empty_cache(pages, page, kv_heads, D, dt, layout, device)

        def randn(*shape):
            return torch.randn(shape, generator=g, device=device, dtype=torch.float32)

        perm = torch.randperm(pages, generator=g, device=device).cpu().tolist()
        table = torch.full((B, blocks), -7, dtype=torch.int32)     # unused entries are no pages
        at = 0
        self.k64, self.v64 = [], []
        sbits = self.scales.view(torch.int16)
        for b in range(B):
            for i in range(used[b]):
                table[b, i] = perm[at + i]
            at += used[b]
            if not fill:
                continue
            # keys with a level of their own per head, some heads of one sign
            k = (randn(kl[b], kv_heads, D) * spread + randn(kv_heads, 1)).to(dt)
            v = (randn(kl[b], kv_heads, D) * torch.exp2(randn(kl[b], kv_heads, 1) * 2)).to(dt)
            both = []
            for x in (k, v):
                c, s, z = quantize(x)
                both.append((pack(c), patterns(s, z, dt)))
            pats = torch.cat([both[0][1], both[1][1]], -1).view(torch.int16)
            for i in range(used[b]):
                n = min(page, kl[b] - i * page)
                rows = slice(i * page, i * page + n)
                self.k_cache[table[b, i], :n] = both[0][0][rows]
                self.v_cache[table[b, i], :n] = both[1][0][rows]
                sbits[table[b, i], :n] = pats[rows]
            self.k64.append(values(*both[0]))
            self.v64.append(values(*both[1]))
        cu = [0]
        for n in ql:
            cu.append(cu[-1] + n)
        self.T = cu[-1]
        self.table = table.to(device)
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor(kl, dtype=torch.int32, device=device)
        self.q = (randn(self.T, q_heads, D) * 1.5 * spread).to(dt)

    def args(self):
        return self.k_cache, self.v_cache, self.scales, self.table, self.cu_q, self.kv_len


def steps15(v):
    """At least 15 s of every value's group: 2.5 times the group's largest value."""
    return 2.5 * v.unflatten(-1, (-1, GROUP)).abs().amax(-1, keepdim=True).expand(-1, -1, GROUP).flatten(-2)


def attention4(bt, scale=None, causal=True, window=0, sinks=0):
    """out, lse in fp64, and per element bounds of the kernels' error:

    out: u |out| (its rounding) + (u + 2^-14) sum p |V| / l: every weight is rounded once
    to 16 bits (u at most), and its own fp32 error stays below 2^-14; and the output is the
    difference of two fp32 sums, of weights times 15 s at most, which grow by 16 keys
    at a time and are joined from a few parts: 2 (kv / 16 + 16) 2^-22 sum p 15 s / l (a value
    may be zero where s is large).  15 s <= 2.5 max |V| over the group: s is (hi - lo) / 15
    times 9 / 8 at most, and the largest of |lo| and |hi|, half of hi - lo at least, is met
    within s / 2.
    Codes are subnormal fp16 operands, c 2^-24, and the matrix instructions align a product by
    its operands' exponent fields, 2^-14 for a subnormal one: what it keeps, 24 bits below
    that, ends at 2^-14 of a step times the largest weight of 16.  Sixteen products are cut
    so, in both sums: 2 * 16 * 2^-14 sum p s / l at most, and s <= max |V| / 6.
    lse: a score is a sum of D fp32 products of queries and codes, each below 15 s |q|, so
    2^-23 D sum 15 s |q| scale at most; for the cut, D 2^-14 s max |q| scale; and the sum and the
    logarithm add a few units of 2^-23."""
    scale = bt.D ** -0.5 if scale is None else scale
    dev = bt.q.device
    out = torch.zeros((bt.T, bt.hq, bt.D), dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    lse = torch.full((bt.T, bt.hq), -math.inf, dtype=torch.float64, device=dev)
    ltol = torch.zeros_like(lse)
    grp, at, u = bt.hq // bt.hk, 0, U[bt.dt]
    for b, (n, kv) in enumerate(zip(bt.ql, bt.kl)):
        p = torch.arange(kv - n, kv, device=dev)[:, None]
        j = torch.arange(kv, device=dev)[None, :]
        see = torch.ones((n, kv), dtype=torch.bool, device=dev)
        if causal:
            see &= j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
        any_key = see.any(1)
        for h in range(bt.hq):
            if n == 0 or kv == 0:
                continue
            q = bt.q[at:at + n, h].double()
            k, v = bt.k64[b][:, h // grp], bt.v64[b][:, h // grp]
            s = (q @ k.T * scale).masked_fill(~see, -math.inf)
            ls = torch.logsumexp(s, 1)
            w = torch.exp(s - ls[:, None].masked_fill(~any_key[:, None], 0.0))
            o = w @ v
            out[at:at + n, h] = o
            tol[at:at + n, h] = u * o.abs() + (u + 2.0 ** -14) * (w @ v.abs()) + 1e-7
            tol[at:at + n, h] += (kv / 8 + 32) * 2.0 ** -22 * (w @ steps15(v)) + 2.0 ** -9 * (w @ steps15(v)) / 15
            lse[at:at + n, h] = ls
            big = (q.abs() @ steps15(k).T * scale).masked_fill(~see, 0.0).amax(1)
            cut = (q.abs().amax(1)[:, None] * steps15(k).amax(1) / 15 * scale).masked_fill(~see, 0.0).amax(1)
            ltol[at:at + n, h] = bt.D * (2.0 ** -23 * big + 2.0 ** -14 * cut) + 2.0 ** -20 * (1 + ls.abs().nan_to_num(posinf=0.0))
        at += n
    return out, tol, lse, ltol


def normed(x, weight, eps):
    """Heads divided by the root of their mean square, times weights, in fp64."""
    x = x.double()
    return x if weight is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()


def positions(bt):
    t = torch.arange(bt.T, device=bt.q.device)
    seq = torch.searchsorted(bt.cu_q[1:].long().contiguous(), t, right=True)
    return seq, bt.kv_len.long()[seq] - (bt.cu_q.long()[seq + 1] - t)


__all__ = ["Batch4", "attention4", "empty_cache", "normed", "pack", "patterns", "positions", "quantize", "rotate",
           "unpack", "values"]
