"""Plain 64-bit forms of the paged cache operators, and batches to test them on
(host-side; shared by the GPU tests)."""
import math

import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
# unit roundoff of the 16-bit types: half a unit in the last place of 8 / 11
# significant bits
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class Batch:
    """A cache and a batch of sequences with `ql` new tokens and `kl` keys (the new
    ones included).  Slots that belong to no key hold NaN."""

    def __init__(self, ql, kl, q_heads, kv_heads, D, dtype="bf16", page=16, layout="hnd", seed=0, device="cuda",
                 spread=1.0, extra_blocks=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        dt = TYPES[dtype]
        self.ql, self.kl, self.hq, self.hk, self.D, self.page, self.dt = ql, kl, q_heads, kv_heads, D, page, dt
        B = len(ql)
        used = [-(-n // page) for n in kl]
        blocks = max(used + [1]) + extra_blocks
        pages = sum(used) + 2

        def randn(*shape):
            return torch.randn(shape, generator=g, device=device, dtype=torch.float32)

        def cache():
            if layout == "hnd":
                return torch.full((pages, kv_heads, page, D), float("nan"), device=device, dtype=dt).permute(0, 2, 1, 3)
            if layout == "nhd":
                return torch.full((pages, page, kv_heads, D), float("nan"), device=device, dtype=dt)
            # rows with room between them
            return torch.full((pages, page, kv_heads, D + 24), float("nan"), device=device, dtype=dt)[..., 8:8 + D]

        self.k_cache, self.v_cache = cache(), cache()
        perm = torch.randperm(pages, generator=g, device=device).cpu().tolist()
        table = torch.full((B, blocks), -7, dtype=torch.int32)     # unused entries are no pages
        at = 0
        self.k64, self.v64 = [], []
        for b in range(B):
            for i in range(used[b]):
                table[b, i] = perm[at + i]
            at += used[b]
            k = (randn(kl[b], kv_heads, D) * spread).to(dt)
            v = randn(kl[b], kv_heads, D).to(dt)
            for i in range(used[b]):
                n = min(page, kl[b] - i * page)
                self.k_cache[table[b, i], :n] = k[i * page:i * page + n]
                self.v_cache[table[b, i], :n] = v[i * page:i * page + n]
            self.k64.append(k.double())
            self.v64.append(v.double())
        cu = [0]
        for n in ql:
            cu.append(cu[-1] + n)
        self.T = cu[-1]
        self.table = table.to(device)
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor(kl, dtype=torch.int32, device=device)
        self.q = (randn(self.T, q_heads, D) * 1.5 * spread).to(dt)

    def args(self):
        return self.k_cache, self.v_cache, self.table, self.cu_q, self.kv_len


def attention(bt, scale=None, causal=True, window=0):
    """out, lse in fp64, and per element bounds of the kernels' error:

    out: u |out| (its rounding) + (u + 2^-14) sum p |V| / l: every weight is rounded
    once to 16 bits (u), and its own fp32 error stays below 2^-14 (scores of a few
    tens, so 2^-23 D |s| and the exponential's 2^-22).
    lse: a score is a sum of D fp32 products, 2^-23 D sum |q k| scale at most, and
    the sum and the logarithm add a few units of 2^-23."""
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
            see &= j > p - window
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
            lse[at:at + n, h] = ls
            big = (q.abs() @ k.abs().T * scale).masked_fill(~see, 0.0).amax(1)
            ltol[at:at + n, h] = bt.D * 2.0 ** -23 * big + 2.0 ** -20 * (1 + ls.abs().nan_to_num(posinf=0.0))
        at += n
    return out, tol, lse, ltol


def rotate(x, pos, cos_sin, interleaved):
    """Rotary positions in fp64: x [tokens][heads][D], pos [tokens]."""
    x = x.double().clone()
    if cos_sin is None:
        return x
    rot = cos_sin.shape[1]
    c = cos_sin[pos, :rot // 2].double()[:, None]
    s = cos_sin[pos, rot // 2:].double()[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2].clone(), x[..., 1:rot:2].clone()
        x[..., 0:rot:2], x[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2].clone(), x[..., rot // 2:rot].clone()
        x[..., :rot // 2], x[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return x


def cos_sin_table(length, rot, device="cuda"):
    f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device=device) * 2 / rot)
    a = torch.arange(length, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()
