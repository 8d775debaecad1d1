"""Measured cases of the paged key/value cache operators: qmm_kv_append (rotate
and store new keys and values) and qmm_paged_attn (attention of new tokens over
the cache).

`run` computes an operator in its plain form (torch operations in 32 bits,
rounded once) where `own` is false, and calls the library where it is true.
`exact` computes the same from the definition in 64 bits.

Sequence b owns tokens cu_q[b] .. cu_q[b+1] of the batch; kv_len[b] counts its
keys with the new ones, so token t sits at position kv_len[b] - (cu_q[b+1] - t).
Key j is slot j % page of page block_table[b][j // page].
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases -----------------------------------------------------------------
def _case(name, op, **kw):
    c = dict(name=name, op=op, dtype="bf16", batch=1, q_lo=1, q_hi=1, kv_lo=1, kv_hi=1, q_heads=32, kv_heads=8,
             head_dim=128, page=16, layout="hnd", spread=1)
    if op == "append":
        c.update(rot=128, interleaved=False)
    else:
        c.update(causal=True, window=0, lse=False)
    c.update(kw)
    return c


def listed():
    return [
        # one token of one conversation: a launch's latency
        _case("append_1_token", "append", kv_lo=700, kv_hi=700),
        # a decode step of 64 conversations
        _case("append_64_decode", "append", dtype="f16", batch=64, kv_lo=100, kv_hi=4096, interleaved=True),
        # ragged prompt chunks, small heads of which half is rotated, cache with the heads innermost
        _case("append_ragged_chunks", "append", batch=5, q_lo=1, q_hi=777, kv_lo=800, kv_hi=2048, q_heads=24,
              kv_heads=6, head_dim=64, rot=32, page=32, layout="nhd"),
        # a long prompt in one piece
        _case("append_8192_prompt", "append", batch=1, q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, q_heads=64,
              page=64),
        # one token over a short conversation: latency of the call
        _case("attn_1_token_517", "attn", kv_lo=517, kv_hi=517),
        # a decode step of 64 conversations of mixed length
        _case("attn_64_decode", "attn", dtype="f16", batch=64, kv_lo=300, kv_hi=4096),
        # one token over a very long document, with the log sums
        _case("attn_1_token_131072", "attn", kv_lo=131072, kv_hi=131072, page=64, lse=True),
        # every head with keys of its own, small heads, heads innermost in the cache
        _case("attn_16_decode_mha", "attn", dtype="f16", batch=16, kv_lo=1000, kv_hi=2048, q_heads=32, kv_heads=32,
              head_dim=64, page=32, layout="nhd"),
        # checking five drafted tokens of each of eight conversations
        _case("attn_8_drafts", "attn", batch=8, q_lo=5, q_hi=5, kv_lo=2000, kv_hi=8192, q_heads=64),
        # the next 512 tokens of a long prompt
        _case("attn_512_chunk_16384", "attn", q_lo=512, q_hi=512, kv_lo=16384, kv_hi=16384),
        # chunks of several prompts at once, a window of 1000 keys, odd lengths
        _case("attn_ragged_window", "attn", dtype="f16", batch=7, q_lo=33, q_hi=699, kv_lo=700, kv_hi=4001,
              q_heads=28, kv_heads=4, head_dim=64, window=1000, lse=True),
        # a long prompt in one piece
        _case("attn_8192_prompt", "attn", q_lo=8192, q_hi=8192, kv_lo=8192, kv_hi=8192, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: either operator, single tokens or chunks, sizes spread over their logarithm."""
    kv_heads = rng.choice([1, 2, 4, 6, 8, 16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8) if g * kv_heads <= 64])
    c = dict(op=rng.choice(["append", "attn", "attn"]), dtype=rng.choice(["bf16", "f16"]), kv_heads=kv_heads,
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
    else:
        c["causal"] = rng.random() < 0.8
        c["window"] = rng.choice([0, 0, _log_int(rng, 1, 4096)]) if c["causal"] else 0
        c["lse"] = rng.random() < 0.5
    return c


def _lengths(case):
    """(new tokens, keys) of every sequence, by the case alone; the first has the most keys."""
    r = random.Random(case["spread"])
    ql = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    kl = [r.randint(max(case["kv_lo"], n), case["kv_hi"]) for n in ql]
    kl[0] = case["kv_hi"]
    return ql, kl


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

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    def cache():   # the pool is full of other and of older keys; logical order [page][slot][head][D]
        if case["layout"] == "hnd":
            return normal(pages, hk, P, D).permute(0, 2, 1, 3)
        return normal(pages, P, hk, D)

    # pages are handed out in no order
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32).cpu()
    table = torch.zeros((B, blocks), dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :used[b]] = perm[at:at + used[b]]
        at += used[b]
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(ql), 0)
    s = dict(case=case, k_cache=cache(), v_cache=cache(), block_table=table.to(dev), cu_q=cu.to(dev),
             kv_len=torch.tensor(kl, dtype=torch.int32, device=dev), max_q=max(ql), max_kv=max(kl), T=T)
    # the fused output of the qkv product; queries, keys and values are views of it
    qkv = normal(T, hq + 2 * hk, D)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    if case["op"] == "append":
        rot = case["rot"]
        s["cos_sin"] = None
        if rot:
            freq = 10000.0 ** (-torch.arange(rot // 2, device=dev, dtype=torch.float64) * 2 / rot)
            ang = torch.arange(max(kl), device=dev, dtype=torch.float64)[:, None] * freq
            s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    else:
        s["q"] = s["q"] * 2    # scores of a few units: some keys matter more than others
        s["scale"] = 1.0 / math.sqrt(D)
    return s


# ---- the operators -----------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        import bit_weight_quantized_gb300 as q
        if c["op"] == "append":
            qr = q.qmm_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_q"],
                                 s["kv_len"], q=s["q"], cos_sin=s["cos_sin"], interleaved=c["interleaved"])
            return {"q": qr, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        r = q.qmm_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_q"], s["kv_len"],
                             s["max_q"], s["max_kv"], scale=s["scale"], causal=c["causal"], window=c["window"],
                             return_lse=c["lse"])
        return {"out": r[0], "lse": r[1]} if c["lse"] else {"out": r}
    return _append_plain(s) if c["op"] == "append" else _attn_plain(s)


def _token_places(s):
    """Sequence and position of every token."""
    t = torch.arange(s["T"], device=s["cu_q"].device)
    cu = s["cu_q"].long()
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return t, seq, s["kv_len"].long()[seq] - (cu[seq + 1] - t)


def _rotated(x, cos, sin, rot, interleaved):
    x = x.float()
    if rot == 0:
        return x
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)


def _append_plain(s):
    c, dt = s["case"], s["k_cache"].dtype
    rot, P = c["rot"], c["page"]
    _, seq, pos = _token_places(s)
    page, slot = s["block_table"].long()[seq, pos // P], pos % P
    cos = sin = None
    if rot:
        cs = s["cos_sin"][pos][:, None, :]
        cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    s["k_cache"][page, slot] = _rotated(s["k"], cos, sin, rot, c["interleaved"]).to(dt)
    s["v_cache"][page, slot] = s["v"]
    return {"q": _rotated(s["q"], cos, sin, rot, c["interleaved"]).to(dt), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _attn_plain(s):
    c = s["case"]
    q, P, D = s["q"], c["page"], c["head_dim"]
    hq, hk = c["q_heads"], c["kv_heads"]
    grp, mq, mk = hq // hk, s["max_q"], s["max_kv"]
    dev = q.device
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    B = kv.numel()
    # every sequence padded to the longest: queries [B][hk][grp * mq][D], keys and values [B][hk][mk][D]
    ti = torch.clamp(cu[:-1, None] + torch.arange(mq, device=dev), max=s["T"] - 1)
    qp = q[ti].float().view(B, mq, hk, grp, D).permute(0, 2, 3, 1, 4).reshape(B, hk, grp * mq, D)
    pages = s["block_table"].long()[:, :-(-mk // P)]
    kp = s["k_cache"][pages].reshape(B, -1, hk, D)[:, :mk].permute(0, 2, 1, 3).float()
    vp = s["v_cache"][pages].reshape(B, -1, hk, D)[:, :mk].permute(0, 2, 1, 3).float()
    sc = torch.matmul(qp, kp.transpose(2, 3)) * s["scale"]
    pos = kv[:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(mq, device=dev)         # [B][mq]
    j = torch.arange(mk, device=dev)
    see = (j < kv[:, None, None]).expand(B, mq, mk)
    if c["causal"]:
        see = see & (j <= pos[..., None])
    if c["window"]:
        see = see & (j > pos[..., None] - c["window"])
    see = see[:, None, None].expand(B, 1, grp, mq, mk).reshape(B, 1, grp * mq, mk)
    sc = sc.masked_fill(~see, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(sc - m0)
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
    if case["op"] == "append":
        rows = T * (hq + 2 * hk) * D * 2
        return {"bytes": 2 * rows + min(T, max(kl)) * case["rot"] * 4 + 4 * (T + 2 * len(ql)),
                "flops": 3 * T * (hq + hk) * case["rot"]}
    pairs = keys = 0
    for n, k in zip(ql, kl):
        w = case["window"] or k
        first = k - n   # position of the first new token
        if case["causal"]:
            # row at position p sees min(p + 1, w) keys
            full = max(0, min(n, w - first))                    # rows that see p + 1 keys
            pairs += full * first + full * (full + 1) // 2 + (n - full) * w
            keys += k - max(0, first - w + 1)
        else:
            pairs += n * k
            keys += k
    return {"bytes": 2 * keys * hk * D * 2 + 2 * T * hq * D * 2 + (4 * T * hq if case["lse"] else 0),
            "flops": 4 * D * hq * pairs}


# ---- the definition in 64 bits -----------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    ql, kl = _lengths(case)
    P, D, hq, hk = case["page"], case["head_dim"], case["q_heads"], case["kv_heads"]
    table = s["block_table"].cpu().tolist()
    if case["op"] == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        qo = s["q"].double()
        kn = s["k"].double()
        rot, at = case["rot"], 0
        for b, (n, kv) in enumerate(zip(ql, kl)):
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
            done = 0
            while done < n:   # page by page
                p = kv - n + done
                take = min(n - done, P - p % P)
                page = table[b][p // P]
                kc[page, p % P:p % P + take] = kn[at + done:at + done + take]
                vc[page, p % P:p % P + take] = s["v"][at + done:at + done + take].double()
                done += take
            at += n
        return {"q": qo, "k_cache": kc, "v_cache": vc}
    if work(case)["flops"] > 2e12:
        return None
    out = torch.zeros((s["T"], hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], hq), float("-inf"), dtype=torch.float64, device="cuda")
    grp, at = hq // hk, 0
    for b, (n, kv) in enumerate(zip(ql, kl)):
        ids = torch.tensor(table[b][:-(-kv // P)], device="cuda", dtype=torch.long)
        p = torch.arange(kv - n, kv, device="cuda")[:, None]
        j = torch.arange(kv, device="cuda")[None, :]
        hidden = torch.zeros((n, kv), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= j > p
        if case["window"]:
            hidden |= j <= p - case["window"]
        for h in range(hk):
            k = s["k_cache"][ids, :, h].reshape(-1, D)[:kv].double()
            v = s["v_cache"][ids, :, h].reshape(-1, D)[:kv].double()
            for g in range(h * grp, (h + 1) * grp):
                a = (s["q"][at:at + n, g].double() @ k.T) * s["scale"]
                a = a.masked_fill(hidden, float("-inf"))
                ls = torch.logsumexp(a, 1)
                out[at:at + n, g] = torch.nan_to_num(torch.exp(a - ls[:, None])) @ v
                lse[at:at + n, g] = ls
        at += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
