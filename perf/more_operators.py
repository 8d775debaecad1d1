"""Measured cases of the 4-bit paged key/value cache operators: qmm_kv4_append (norm,
rotate, quantise and store new keys and values), qmm_kv4_read (the values that keys of
the cache stand for) and qmm_kv4_attn (attention of new tokens over the cache, with a
window and first tokens that stay visible).

`run` computes an operator in its plain form (torch operations in 32 bits,
rounded once) where `own` is false, and calls the library where it is true.
`exact` computes the same from the definition in 64 bits.

Sequence b owns tokens cu_q[b] .. cu_q[b+1] of the batch; kv_len[b] counts its
keys with the new ones, so token t sits at position kv_len[b] - (cu_q[b+1] - t).
Key j is slot j % page of page block_table[b][j // page].  64 values of a head share
a scale s and a zero z: a code c stands for (c - z) * s, codes two to a byte, the low
half first.  s has 4 significant bits in bf16 and 7 in f16, z is in the low four bits
of its pattern; a key's scales are those of its key's groups, then of its value's.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_GROUP = 64


# ---- cases -----------------------------------------------------------------
def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", batch=1, q_lo=1, q_hi=1, kv_lo=1, kv_hi=1, q_heads=32, kv_heads=8,
             head_dim=128, page=16, layout="hnd", spread=1)
    if op == "append":
        c.update(rot=128, interleaved=False, norm=False)
    elif op == "attn":
        c.update(causal=True, window=0, sinks=0, lse=False)
    c.update(kw)
    return c


def listed():
    return [
        # one token of one conversation, queries and keys normed: a launch's latency
        _case("append_1_token", "append", kv_lo=700, kv_hi=700, norm=True),
        # a decode step of 64 conversations
        _case("append_64_decode", "append", dtype="f16", batch=64, kv_lo=100, kv_hi=4096, interleaved=True),
        # a long prompt in one piece, queries and keys normed
        _case("append_8192_prompt", "append", q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, q_heads=64, page=64,
              norm=True),
        # the last keys of three conversations taken out of the cache, small heads, heads innermost, odd pages
        _case("read_3_tails", "read", dtype="f16", batch=3, q_lo=5, q_hi=333, kv_lo=400, kv_hi=1001, kv_heads=6,
              q_heads=24, head_dim=64, page=24, layout="nhd"),
        # a whole long document read back, to go on in 16 bits
        _case("read_131072", "read", q_lo=131072, q_hi=131072, kv_lo=131072, kv_hi=131072, page=64),
        # one token over a short conversation: latency of the call
        _case("attn_1_token_517", "attn", kv_lo=517, kv_hi=517),
        # a decode step of 64 conversations of mixed length
        _case("attn_64_decode", "attn", dtype="f16", batch=64, kv_lo=300, kv_hi=4096),
        # one token over a very long document, with the log sums
        _case("attn_1_token_131072", "attn", kv_lo=131072, kv_hi=131072, page=64, lse=True),
        # five drafted tokens of each of 24 conversations, a window and four first tokens
        _case("attn_24_drafts_sinks", "attn", batch=24, q_lo=5, q_hi=5, kv_lo=2000, kv_hi=8192, q_heads=64,
              window=2048, sinks=4),
        # the next 512 tokens of a long prompt
        _case("attn_512_chunk_16384", "attn", q_lo=512, q_hi=512, kv_lo=16384, kv_hi=16384),
        # chunks of several prompts at once, small heads, a window and first tokens, odd lengths
        _case("attn_ragged_sinks", "attn", dtype="f16", batch=7, q_lo=33, q_hi=699, kv_lo=700, kv_hi=4001,
              q_heads=28, kv_heads=4, head_dim=64, window=1000, sinks=5, lse=True),
        # a long prompt in one piece
        _case("attn_8192_prompt", "attn", q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, q_heads=64, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: any operator, single tokens or chunks, sizes spread over their logarithm."""
    kv_heads = rng.choice([1, 2, 4, 6, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8) if g * kv_heads <= 64])
    c = dict(op=rng.choice(["append", "read", "attn", "attn"]), dtype=rng.choice(["bf16", "f16"]), kv_heads=kv_heads,
             q_heads=kv_heads * group, head_dim=rng.choice([64, 128]), page=rng.choice([8, 16, 24, 32, 64, 128]),
             layout=rng.choice(["hnd", "nhd"]), spread=rng.randrange(1 << 20))
    if rng.random() < 0.5:      # single tokens
        c["batch"] = _log_int(rng, 1, 96)
        c["q_lo"] = c["q_hi"] = 1
    else:                       # chunks
        c["batch"] = _log_int(rng, 1, 8)
        c["q_hi"] = _log_int(rng, 2, max(2, 4096 // c["batch"]))
        c["q_lo"] = rng.randint(1, c["q_hi"])
    c["kv_hi"] = c["q_hi"] + _log_int(rng, 1, 16384)
    # no more than the listed cases' keys and scores
    while c["batch"] * c["kv_hi"] * c["kv_heads"] * c["head_dim"] > 96 * 1024 * 1024 and c["kv_hi"] > 2 * c["q_hi"]:
        c["kv_hi"] = max(c["q_hi"] + 1, c["kv_hi"] // 2)
    while c["batch"] * c["q_hi"] * c["kv_hi"] * c["q_heads"] > 1 << 30:
        c["q_hi"] = max(1, c["q_hi"] // 2)
        c["q_lo"] = min(c["q_lo"], c["q_hi"])
    c["kv_lo"] = rng.randint(c["q_hi"], c["kv_hi"])
    if c["op"] == "append":
        c["rot"] = rng.choice([0, 32, 64, c["head_dim"]])
        c["interleaved"] = rng.random() < 0.5
        c["norm"] = rng.random() < 0.5
    elif c["op"] == "attn":
        c["causal"] = rng.random() < 0.8
        c["window"] = rng.choice([0, 0, _log_int(rng, 1, 4096)]) if c["causal"] else 0
        c["sinks"] = rng.choice([0, 1, 4, _log_int(rng, 1, 300)]) if c["window"] else 0
        c["lse"] = rng.random() < 0.5
    elif rng.random() < 0.5:    # read back: whole sequences, or what is new
        c["q_lo"] = c["kv_lo"]
        c["q_hi"] = c["kv_hi"]
    return c


def _lengths(case):
    """(new tokens, keys) of every sequence, by the case alone; the first has the most keys."""
    r = random.Random(case["spread"])
    ql = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    kl = [r.randint(max(case["kv_lo"], n), case["kv_hi"]) for n in ql]
    kl[0] = case["kv_hi"]
    return ql, kl


# ---- the format ----------------------------------------------------------------
def _quantised(x):
    """16-bit values [..., D] -> codes uint8 [..., D / 2], scales with their zeros [..., D / 64]."""
    dt, D = x.dtype, x.shape[-1]
    g = x.float().unflatten(-1, (D // _GROUP, _GROUP))
    lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
    # (a tensor divides: torch multiplies by a number's rounded reciprocal, which misses quotients on the grid)
    s = (hi * 0.5 - lo * 0.5) / torch.full_like(hi, 7.5)
    low = (1 << 20) - 1 if dt == torch.bfloat16 else (1 << 17) - 1     # bits of a 32-bit pattern that s does not have
    up = ((s.view(torch.int32) + low) & ~low).view(torch.float32)
    if dt == torch.float16:     # below the type's normal numbers: whole steps of 2^-20
        up = torch.where(s < 2.0 ** -14, torch.ceil(s * 2.0 ** 20) * 2.0 ** -20, up)
    s = torch.where(torch.isfinite(s), up, torch.full_like(s, float("nan")))
    d = torch.where(s == 0, torch.ones_like(s), s)
    z = torch.round(-lo / d).clamp(0, 15)
    c = (torch.round(g / d[..., None]) + z[..., None]).clamp(0, 15)
    v, most = (c - z[..., None]) * s[..., None], torch.finfo(dt).max
    c = c - (v > most).float() + (v < -most).float()       # the values stay finite
    c, z = torch.nan_to_num(c).to(torch.uint8).flatten(-2), torch.nan_to_num(z).to(torch.int16)
    bits = torch.where(torch.isnan(s), torch.full_like(z, 0x7ff0), (s.to(dt).view(torch.int16) & -16) | z)
    return c[..., 0::2] | (c[..., 1::2] << 4), bits.view(dt)


def _values(codes, scales):
    """Codes [..., D / 2] and scales [..., D / 64] -> the values they stand for, fp32 [..., D]."""
    bits = scales.view(torch.int16)
    s, z = (bits & -16).view(scales.dtype).float(), (bits & 15).float()
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return ((c.unflatten(-1, (-1, _GROUP)) - z[..., None]) * s[..., None]).flatten(-2)


# ---- inputs ----------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt, D, P = _TYPES[case["dtype"]], case["head_dim"], case["page"]
    hq, hk = case["q_heads"], case["kv_heads"]
    ql, kl = _lengths(case)
    T, B = sum(ql), len(ql)
    blocks = max(-(-n // P) for n in kl)
    used = [-(-n // P) for n in kl]
    pages = sum(used) + 3
    inner = (hk, P) if case["layout"] == "hnd" else (P, hk)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    def order(t):   # logical order [page][slot][head][...]
        return t.permute(0, 2, 1, 3) if case["layout"] == "hnd" else t

    # the pool is full of other and of older keys; channels of the keys have levels of their own
    level = 1 + 0.5 * torch.randn(D, generator=gen, device=dev)
    k_cache, v_cache = (torch.empty((pages, *inner, D // 2), dtype=torch.uint8, device=dev) for _ in range(2))
    scales = torch.empty((pages, *inner, 2 * D // _GROUP), dtype=dt, device=dev)
    step = max(1, (64 << 20) // (P * hk * D))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        k_cache[i:i + n], scales[i:i + n, ..., :D // _GROUP] = _quantised((normal(n, *inner, D) * level).to(dt))
        v_cache[i:i + n], scales[i:i + n, ..., D // _GROUP:] = _quantised(normal(n, *inner, D))
    # pages are handed out in no order
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).cpu()
    table = torch.zeros((B, blocks), dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :used[b]] = perm[at:at + used[b]]
        at += used[b]
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(ql), 0)
    s = dict(case=case, k_cache=order(k_cache), v_cache=order(v_cache), scales=order(scales), block_table=table.to(dev),
             cu_q=cu.to(dev), kv_len=torch.tensor(kl, dtype=torch.int32, device=dev), max_q=max(ql), max_kv=max(kl), T=T)
    if case["op"] == "read":
        return s
    # the fused output of the qkv product; queries, keys and values are views of it
    qkv = normal(T, hq + 2 * hk, D)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    if case["op"] == "append":
        rot = case["rot"]
        s["cos_sin"] = s["q_norm"] = s["k_norm"] = None
        if rot:
            freq = 10000.0 ** (-torch.arange(rot // 2, device=dev, dtype=torch.float64) * 2 / rot)
            ang = torch.arange(max(kl), device=dev, dtype=torch.float64)[:, None] * freq
            s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        if case["norm"]:
            s["q_norm"], s["k_norm"] = (1 + 0.2 * normal(2, D)).to(dt).contiguous()
            s["eps"] = 1e-6
    else:
        s["q"] = s["q"] * 2    # scores of a few units: some keys matter more than others
        s["scale"] = 1.0 / math.sqrt(D)
    return s


# ---- the operators -----------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        import bit_weight_quantized_gb300 as q
        cache = s["k_cache"], s["v_cache"], s["scales"], s["block_table"], s["cu_q"], s["kv_len"]
        if c["op"] == "attn":
            r = q.qmm_kv4_attn(s["q"], *cache, s["max_q"], s["max_kv"], scale=s["scale"], causal=c["causal"],
                               window=c["window"], sinks=c["sinks"], return_lse=c["lse"])
            return {"out": r[0], "lse": r[1]} if c["lse"] else {"out": r}
        r = {}
        if c["op"] == "append":
            norm = dict(q_norm=s["q_norm"], k_norm=s["k_norm"], eps=s["eps"]) if c["norm"] else {}
            r["q"] = q.qmm_kv4_append(s["k"], s["v"], *cache, q=s["q"], cos_sin=s["cos_sin"],
                                      interleaved=c["interleaved"], **norm)
        # (after an append: what it stored, as the values it stands for)
        r["k"], r["v"] = q.qmm_kv4_read(*cache, s["T"])
        return r
    if c["op"] == "attn":
        return _attn_plain(s)
    r = _append_plain(s) if c["op"] == "append" else {}
    return {**r, **_read_plain(s)}


def _token_places(s):
    """Sequence and position of every token."""
    t = torch.arange(s["T"], device=s["cu_q"].device)
    cu = s["cu_q"].long()
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return t, seq, s["kv_len"].long()[seq] - (cu[seq + 1] - t)


def _turned(x, weight, eps, cos, sin, rot, interleaved):
    """Normed (weight not None) and rotated, in fp32."""
    x = x.float()
    if weight is not None:
        r = torch.rsqrt(x.double().square().mean(-1, keepdim=True) + eps).float()
        x = x * r * weight.float()
    if rot == 0:
        return x
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)


def _append_plain(s):
    c, dt = s["case"], s["scales"].dtype
    rot, P = c["rot"], c["page"]
    _, seq, pos = _token_places(s)
    page, slot = s["block_table"].long()[seq, pos // P], pos % P
    cos = sin = None
    if rot:
        cs = s["cos_sin"][pos][:, None, :]
        cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    eps = s.get("eps", 0.0)
    kc, ks = _quantised(_turned(s["k"], s["k_norm"], eps, cos, sin, rot, c["interleaved"]).to(dt))
    vc, vs = _quantised(s["v"])
    s["k_cache"][page, slot] = kc
    s["v_cache"][page, slot] = vc
    s["scales"][page, slot] = torch.cat([ks, vs], -1)
    return {"q": _turned(s["q"], s["q_norm"], eps, cos, sin, rot, c["interleaved"]).to(dt)}


def _read_plain(s):
    c, dt = s["case"], s["scales"].dtype
    P, half = c["page"], c["head_dim"] // _GROUP
    _, seq, pos = _token_places(s)
    page, slot = s["block_table"].long()[seq, pos // P], pos % P
    sc = s["scales"][page, slot]
    return {"k": _values(s["k_cache"][page, slot], sc[..., :half].contiguous()).to(dt),
            "v": _values(s["v_cache"][page, slot], sc[..., half:].contiguous()).to(dt)}


def _attn_plain(s):
    c = s["case"]
    q, P, D = s["q"], c["page"], c["head_dim"]
    hq, hk = c["q_heads"], c["kv_heads"]
    grp, mq, mk, half = hq // hk, s["max_q"], s["max_kv"], D // _GROUP
    dev = q.device
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    B = kv.numel()
    # every sequence padded to the longest: queries [B][hk][grp * mq][D], keys and values [B][hk][mk][D]
    ti = torch.clamp(cu[:-1, None] + torch.arange(mq, device=dev), max=s["T"] - 1)
    qp = q[ti].float().view(B, mq, hk, grp, D).permute(0, 2, 3, 1, 4).reshape(B, hk, grp * mq, D)
    pages = s["block_table"].long()[:, :-(-mk // P)]
    sc = s["scales"][pages].reshape(B, -1, hk, 2 * half)[:, :mk].permute(0, 2, 1, 3)
    kp = _values(s["k_cache"][pages].reshape(B, -1, hk, D // 2)[:, :mk].permute(0, 2, 1, 3), sc[..., :half].contiguous())
    vp = _values(s["v_cache"][pages].reshape(B, -1, hk, D // 2)[:, :mk].permute(0, 2, 1, 3), sc[..., half:].contiguous())
    x = torch.matmul(qp, kp.transpose(2, 3)) * s["scale"]
    pos = kv[:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(mq, device=dev)         # [B][mq]
    j = torch.arange(mk, device=dev)
    see = (j < kv[:, None, None]).expand(B, mq, mk)
    if c["causal"]:
        see = see & (j <= pos[..., None])
    if c["window"]:
        see = see & ((j > pos[..., None] - c["window"]) | (j < c["sinks"]))
    see = see[:, None, None].expand(B, 1, grp, mq, mk).reshape(B, 1, grp * mq, mk)
    x = x.masked_fill(~see, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m0)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, vp) / torch.where(l > 0, l, torch.ones_like(l))
    t, seq, _ = _token_places(s)
    i = t - cu[seq]
    o = o.view(B, hk, grp, mq, D).permute(0, 3, 1, 2, 4).reshape(B, mq, hq, D)[seq, i]
    r = {"out": o.to(q.dtype)}
    if c["lse"]:
        r["lse"] = (m0 + torch.log(l)).view(B, hq, mq).permute(0, 2, 1)[seq, i]
    return r


# ---- what a pass cannot do without -------------------------------------------------
def work(case):
    ql, kl = _lengths(case)
    T, D, hq, hk = sum(ql), case["head_dim"], case["q_heads"], case["kv_heads"]
    key = hk * (D + 4 * D // _GROUP)      # bytes of a key and its value, all heads
    if case["op"] == "read":
        return {"bytes": T * (key + 4 * hk * D) + 4 * (-(-T // case["page"]) + 2 * len(ql)), "flops": 4 * T * hk * D}
    if case["op"] == "append":
        rows = T * (hq + 2 * hk) * D * 2
        # rows in; queries, the cache's and the read back values out
        return {"bytes": 2 * rows + T * key + min(T, max(kl)) * case["rot"] * 4 + 4 * (T + 2 * len(ql)),
                "flops": T * (3 * (hq + hk) * case["rot"] + (4 * (hq + hk) * D if case["norm"] else 0) + 8 * hk * D)}
    pairs = keys = 0
    for n, k in zip(ql, kl):
        w = case["window"] or k
        first = k - n   # position of the first new token
        if case["causal"]:
            # row at position p sees min(p + 1, w) keys, and the first ones before those
            full = max(0, min(n, w - first))                    # rows that see p + 1 keys
            pairs += full * first + full * (full + 1) // 2 + (n - full) * w
            pairs += sum(min(case["sinks"], max(0, p + 1 - w)) for p in range(first, k))
            keys += k - max(0, first - w + 1) + min(case["sinks"], max(0, first - w + 1))
        else:
            pairs += n * k
            keys += k
    return {"bytes": keys * key + 2 * T * hq * D * 2 + (4 * T * hq if case["lse"] else 0),
            "flops": 4 * D * hq * pairs}


# ---- the definition in 64 bits -----------------------------------------------------
def _exact_scale(x, bits, least):
    """The smallest number of so many significant bits that is not below x (not below `least`'s multiples)."""
    m, e = torch.frexp(x)
    # (torch.ldexp multiplies by a power of two computed in 32 bits, on the GPU not exactly)
    y = torch.ceil(m * 2.0 ** bits) * ((e.long() - bits + 1023) << 52).view(torch.float64)
    return torch.where(y < 2.0 ** bits * least, torch.ceil(x / least) * least, y)


def _exact_stored(x, dt):
    """What the cache holds for 64-bit values x: rounded to the type, then to codes."""
    x = x.to(dt).double()
    for g in range(0, x.shape[-1], _GROUP):
        v = x[..., g:g + _GROUP]
        lo, hi = torch.clamp(v.amin(-1, keepdim=True), max=0), torch.clamp(v.amax(-1, keepdim=True), min=0)
        s = _exact_scale((hi - lo) / torch.full_like(hi, 15.0), 4 if dt == torch.bfloat16 else 7, 2.0 ** -129 if dt == torch.bfloat16 else 2.0 ** -20)
        s = torch.where(s > 0, s, torch.ones_like(s))
        z = torch.clamp(torch.round(-lo / s), 0, 15)
        x[..., g:g + _GROUP] = (torch.clamp(torch.round(v / s) + z, 0, 15) - z) * s
    return x


def _exact_read(s, b, lo, hi, h):
    """Keys lo .. hi - 1 of sequence b, head h, and their values, in 64 bits."""
    c = s["case"]
    P, D = c["page"], c["head_dim"]
    ids = s["block_table"][b, lo // P:-(-hi // P)].long()
    sl = slice(lo - lo // P * P, hi - lo // P * P)
    raw = s["scales"][ids, :, h].reshape(-1, 2 * D // _GROUP)[sl].contiguous().view(torch.int16).int()
    out = []
    for n, cache in enumerate((s["k_cache"], s["v_cache"])):
        byte = cache[ids, :, h].reshape(-1, D // 2)[sl]
        v = torch.empty((hi - lo, D), dtype=torch.float64, device=byte.device)
        v[:, 0::2], v[:, 1::2] = (byte % 16).double(), (byte // 16).double()
        for g in range(D // _GROUP):
            r = raw[:, n * (D // _GROUP) + g]
            z = r % 16
            scale = (r - z).to(torch.int16).view(s["scales"].dtype).double()
            v[:, g * _GROUP:(g + 1) * _GROUP] = (v[:, g * _GROUP:(g + 1) * _GROUP] - z[:, None]) * scale[:, None]
        out.append(v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    ql, kl = _lengths(case)
    D, hq, hk, dt = case["head_dim"], case["q_heads"], case["kv_heads"], _TYPES[case["dtype"]]
    if case["op"] == "read":
        k = torch.empty((s["T"], hk, D), dtype=torch.float64, device="cuda")
        v, at = torch.empty_like(k), 0
        for b, (n, kv) in enumerate(zip(ql, kl)):
            for h in range(hk):
                k[at:at + n, h], v[at:at + n, h] = _exact_read(s, b, kv - n, kv, h)
            at += n
        return {"k": k, "v": v}
    if case["op"] == "append":
        qo, kn = s["q"].double(), s["k"].double()
        rot, at = case["rot"], 0
        if case["norm"]:
            qo, kn = (x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + s["eps"]) * w.double()
                      for x, w in ((qo, s["q_norm"]), (kn, s["k_norm"])))
        for n, kv in zip(ql, kl):
            rows = slice(at, at + n)
            for x in (qo, kn):
                if not rot:
                    continue
                # a pair (a, b) is the complex number a + i b, turned by cos + i sin
                cs = s["cos_sin"][kv - n:kv].double()
                turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None, :]
                if case["interleaved"]:
                    z = torch.view_as_complex(x[rows, :, :rot].reshape(n, -1, rot // 2, 2).contiguous()) * turn
                    x[rows, :, :rot] = torch.view_as_real(z).reshape(n, -1, rot)
                else:
                    z = torch.complex(x[rows, :, :rot // 2].contiguous(), x[rows, :, rot // 2:rot].contiguous()) * turn
                    x[rows, :, :rot] = torch.cat([z.real, z.imag], -1)
            at += n
        return {"q": qo, "k": _exact_stored(kn, dt), "v": _exact_stored(s["v"].double(), dt)}
    if work(case)["flops"] > 2e12:
        return None
    out = torch.zeros((s["T"], hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], hq), float("-inf"), dtype=torch.float64, device="cuda")
    grp, at = hq // hk, 0
    for b, (n, kv) in enumerate(zip(ql, kl)):
        p = torch.arange(kv - n, kv, device="cuda")[:, None]
        j = torch.arange(kv, device="cuda")[None, :]
        hidden = torch.zeros((n, kv), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= j > p
        if case["window"]:
            hidden |= (j <= p - case["window"]) & (j >= case["sinks"])
        for h in range(hk):
            k, v = _exact_read(s, b, 0, kv, h)
            for g in range(h * grp, (h + 1) * grp):
                a = (s["q"][at:at + n, g].double() @ k.T) * s["scale"]
                a = a.masked_fill(hidden, float("-inf"))
                ls = torch.logsumexp(a, 1)
                out[at:at + n, g] = torch.nan_to_num(torch.exp(a - ls[:, None])) @ v
                lse[at:at + n, g] = ls
        at += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
