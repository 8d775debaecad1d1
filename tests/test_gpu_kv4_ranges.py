"""qmm_kv4_attn where the values' sizes differ widely between keys, between the two groups of a
head and between what the rows of a call see, against a 64-bit form, with the bounds of each
kernel: few query rows multiply codes, many the values themselves."""
import math

import pytest
import torch

from kv4_ref import GROUP, Batch4, pack, patterns, quantize, steps15, values
from paged_ref import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_weight_quantized_gb300 as q
    q.load()
    return q


def store(bt, b, k, v):
    """Sequence b's keys and values (of bt.dt), quantized, into the cache and the 64-bit copies."""
    page, n = bt.page, k.shape[0]
    (ck, sk, zk), (cv, sv, zv) = quantize(k), quantize(v)
    pk, pv = patterns(sk, zk, bt.dt), patterns(sv, zv, bt.dt)
    pats = torch.cat([pk, pv], -1).view(torch.int16)
    sbits = bt.scales.view(torch.int16)
    for i, at in enumerate(bt.table[b, :-(-n // page)].tolist()):
        rows = slice(i * page, min(n, (i + 1) * page))
        m = rows.stop - rows.start
        bt.k_cache[at, :m] = pack(ck[rows])
        bt.v_cache[at, :m] = pack(cv[rows])
        sbits[at, :m] = pats[rows]
    bt.k64[b], bt.v64[b] = values(pack(ck), pk), values(pack(cv), pv)


def reference(bt, few, causal=True, window=0, sinks=0):
    """out and lse in fp64 and bounds of the kernel's error per element.  Weights w = p / l.

    Both: u |out| for the output's rounding; every weight is rounded once to 16 bits, half a unit (few
    rows: fp16, 2^-11; many: the type's, u), and its own fp32 error (scores of a few tens, so 2^-23 D |s|,
    and the exponential's 2^-22) stays below 2^-14, each of sum w |V|.
    Few rows: codes are subnormal operands, of whose products the matrix instructions keep 2^-14 of a
    step s: a score is off by D 2^-14 s max |q| scale at most, which is its weight's and the sum's relative error;
    the output's two sums by 2 * 16 * 2^-14 times the largest w s of 16 keys each, 2^-9 sum w s at most; they
    are differences of fp32 sums of 15 w s, 16 keys at a time: 2 (kv / 16 + 16) 2^-22 sum 15 w s.  Weights
    times scales end at 2^-32 of the largest of their row and group (fp16 from 2^7 down to 2^-25):
    15 kv 2^-32 max w s.
    lse: D 2^-23 sum |q K| scale for fp32 products, the largest score error, a few units of 2^-23."""
    scale = bt.D ** -0.5
    dev = bt.q.device
    out = torch.zeros((bt.T, bt.hq, bt.D), dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    lse, ltol = (torch.full((bt.T, bt.hq), x, dtype=torch.float64, device=dev) for x in (-math.inf, 0.0))
    grp, at, u = bt.hq // bt.hk, 0, U[bt.dt]
    uw = 2.0 ** -11 if few else u
    for b, (n, kv) in enumerate(zip(bt.ql, bt.kl)):
        pos = torch.arange(kv - n, kv, device=dev)[:, None]
        j = torch.arange(kv, device=dev)[None, :]
        see = torch.ones((n, kv), dtype=torch.bool, device=dev)
        if causal:
            see &= j <= pos
        if window:
            see &= (j > pos - window) | (j < sinks)
        for h in range(bt.hq):
            x = bt.q[at:at + n, h].double()
            k, v = bt.k64[b][:, h // grp], bt.v64[b][:, h // grp]
            s = (x @ k.T * scale).masked_fill(~see, -math.inf)
            ls = torch.logsumexp(s, 1)
            w = torch.exp(s - ls[:, None])
            o = w @ v
            t = u * o.abs() + (uw + 2.0 ** -14) * (w @ v.abs())
            big = (x.abs() @ k.abs().T * scale).masked_fill(~see, 0.0).amax(1)
            lt = bt.D * 2.0 ** -23 * big + 2.0 ** -20 * (1 + ls.abs())
            if few:
                step = steps15(v) / 15
                cut = bt.D * 2.0 ** -14 * x.abs().amax(1)[:, None] * (steps15(k) / 15).amax(1) * scale
                off = (w * cut).sum(1, keepdim=True)      # the sum's relative error
                t += (w * cut) @ v.abs() + off * o.abs()
                t += 2.0 ** -9 * (w @ step) + (kv / 8 + 32) * 2.0 ** -22 * 15 * (w @ step)
                most = torch.stack([(w * step[:, c][None]).amax(1) for c in range(0, bt.D, GROUP)], 1)
                t += 15 * kv * 2.0 ** -32 * most.repeat_interleave(GROUP, 1)
                lt += off[:, 0]
            out[at:at + n, h], tol[at:at + n, h], lse[at:at + n, h], ltol[at:at + n, h] = o, t, ls, lt
        at += n
    return out, tol, lse, ltol


def check(q, bt, few=True, **kw):
    got, lse = q.qmm_kv4_attn(bt.q, *bt.args(), max(bt.ql), max(bt.kl), return_lse=True, **kw)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    ref, tol, ls, ltol = reference(bt, few, **kw)
    bad = ~((got.double() - ref).abs() <= tol + 2.0 ** -133)         # (half a step of the smallest bf16 numbers)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs out of bounds, first at {bad.nonzero()[0].tolist()}"
    assert ((lse.double() - ls).abs() <= ltol).all()
    return got


def keys_and_values(bt, b, level, seed=0):
    """Queries with a common direction, keys that lie at `level` [keys] nats along it, normal values."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    sign = torch.where(torch.arange(bt.D, device="cuda") % 3 == 0, -1.0, 1.0)
    lo, hi = sum(bt.ql[:b]), sum(bt.ql[:b + 1])
    rows = torch.randn((hi - lo, bt.hq, bt.D), generator=g, device="cuda")
    bt.q[lo:hi] = (2 * sign + rows / 4).to(bt.dt)
    n = bt.kl[b]
    k = torch.randn((n, bt.hk, bt.D), generator=g, device="cuda") / 2
    k += level[:, None, None] * sign / (2 * bt.D ** 0.5)
    return k, torch.randn((n, bt.hk, bt.D), generator=g, device="cuda")


# Values of the others and factor of the large ones: within the type's numbers.
SIZES = [("bf16", 1.0, 20), ("bf16", 1.0, 24), ("bf16", 1.0, 30), ("bf16", 2.0 ** -60, 100), ("f16", 2.0 ** -8, 20)]
# items in clusters of eight-warp blocks, in a block each, split over all; 4 to 16 rows
FORMS = [([1], [300], (8, 2)), ([2, 1], [2000, 40], (8, 2)), ([1] * 40, [130] * 40, (16, 8)), ([3], [30000], (5, 1))]


# Large values under scores so low that they do not count, or count as much as the others.
@pytest.mark.parametrize("dtype,base,r", SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("nats", [60.0, 17.0])
@pytest.mark.parametrize("where", ["first", "one", "last"])
def test_large_values_under_low_scores(q, dtype, base, r, D, form, nats, where):
    ql, kl, heads = FORMS[form]
    bt = Batch4(ql, kl, *heads, D, dtype, fill=False)
    bt.k64, bt.v64 = [None] * len(ql), [None] * len(ql)
    for b, n in enumerate(kl):
        large = torch.zeros(n, dtype=torch.bool, device="cuda")
        large[{"first": slice(0, 33), "one": slice(n // 2, n // 2 + 1), "last": slice(n - ql[b] - 3, n - ql[b])}[where]] = True
        k, v = keys_and_values(bt, b, torch.where(large, -nats, 0.0), seed=b)
        v = v * base * torch.where(large, 2.0 ** r, 1.0)[:, None, None]
        store(bt, b, k.to(bt.dt), v.to(bt.dt))
    check(q, bt)


# Keys that only some rows of an item see: the last new token's, and those before the window.
@pytest.mark.parametrize("dtype,base,r", SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql,kl,heads", [([4], [300], (8, 2)), ([8, 5], [40, 2000], (4, 2)), ([2], [30000], (16, 2))])
@pytest.mark.parametrize("window,sinks", [(0, 0), (25, 3)])
def test_large_values_under_hidden_keys(q, dtype, base, r, D, ql, kl, heads, window, sinks):
    bt = Batch4(ql, kl, *heads, D, dtype, fill=False)
    bt.k64, bt.v64 = [None] * len(ql), [None] * len(ql)
    for b, n in enumerate(kl):
        k, v = keys_and_values(bt, b, torch.zeros(n, device="cuda"), seed=b)
        v *= base
        v[n - 1] *= 2.0 ** r
        if window:
            v[n - ql[b] - window + 1] *= 2.0 ** r         # the first token's alone
        store(bt, b, k.to(bt.dt), v.to(bt.dt))
    check(q, bt, window=window, sinks=sinks)


# One group of one key: the other group's values keep their bits.
@pytest.mark.parametrize("dtype,base,r", SIZES)
@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("group", [0, 1])
def test_large_values_in_one_group(q, dtype, base, r, form, group):
    ql, kl, heads = FORMS[form]
    bt = Batch4(ql, kl, *heads, 128, dtype, fill=False)
    bt.k64, bt.v64 = [None] * len(ql), [None] * len(ql)
    for b, n in enumerate(kl):
        k, v = keys_and_values(bt, b, torch.zeros(n, device="cuda"), seed=b)
        v *= base
        v[n // 3, :, group * GROUP:(group + 1) * GROUP] *= 2.0 ** r
        store(bt, b, k.to(bt.dt), v.to(bt.dt))
    check(q, bt)


# Scores that rise along the axis while values shrink: the largest part of the sum is taken over again and again.
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rise", [0.4, 3.0, -0.4])
def test_rising_scores_and_shrinking_values(q, dtype, D, rise):
    bt = Batch4([1, 3], [1500, 700], 8, 2, D, dtype, fill=False)
    bt.k64, bt.v64 = [None] * 2, [None] * 2
    for b, n in enumerate(bt.kl):
        j = torch.arange(n, device="cuda")
        part = (j // 32).float()
        k, v = keys_and_values(bt, b, part * rise, seed=b)
        shrink = torch.exp2(-part.clamp(max=20 if dtype == "f16" else 60)) * 2.0 ** (8 if dtype == "f16" else 30)
        store(bt, b, k.to(bt.dt), (v * shrink[:, None, None]).to(bt.dt))
    check(q, bt)


# All values small or large; half of the groups zeros.
@pytest.mark.parametrize("dtype,e", [("bf16", -100), ("bf16", -128), ("bf16", 105), ("f16", -13), ("f16", 12)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_ends_of_the_type(q, dtype, e, D, form):
    ql, kl, heads = FORMS[form]
    bt = Batch4(ql, kl, *heads, D, dtype, fill=False)
    bt.k64, bt.v64 = [None] * len(ql), [None] * len(ql)
    for b, n in enumerate(kl):
        k, v = keys_and_values(bt, b, torch.zeros(n, device="cuda"), seed=b)
        v = (v.double() * 2.0 ** e).to(bt.dt)
        v[::2, :, D - GROUP:] = 0
        store(bt, b, k.to(bt.dt), v)
    check(q, bt)


# Many rows multiply the values themselves: the same sizes, within the 16-bit cache's bounds, and log sums
# that would miss a key that was left out.
@pytest.mark.parametrize("dtype,base,r", SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql,kl,heads,window,sinks", [([300, 133], [700, 140], (8, 2), 0, 0), ([400], [1000], (8, 1), 200, 5),
                                                      ([1030], [2100], (64, 8), 0, 0)])
def test_many_rows(q, dtype, base, r, D, ql, kl, heads, window, sinks):
    bt = Batch4(ql, kl, *heads, D, dtype, fill=False)
    bt.k64, bt.v64 = [None] * len(ql), [None] * len(ql)
    for b, n in enumerate(kl):
        large = torch.arange(n, device="cuda") == n // 2
        k, v = keys_and_values(bt, b, torch.where(large, -40.0, 0.0), seed=b)
        v = v * base * torch.where(large, 2.0 ** r, 1.0)[:, None, None]
        v[n - 1] *= 2.0 ** min(r, 20)
        store(bt, b, k.to(bt.dt), v.to(bt.dt))
    check(q, bt, few=False, window=window, sinks=sinks)


# Scores of ordinary size from sizes at the ends of the type's.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql", [[1], [3]])
@pytest.mark.parametrize("q_e,k_e,scale_e", [(-70, 124, -70), (-110, 120, -29), (100, -110, -1), (-100, -20, 115), (10, -122, 104)])
def test_scores_of_large_and_small_factors(q, D, ql, q_e, k_e, scale_e):
    bt = Batch4(ql, [300], 8, 2, D, "bf16", fill=False)
    bt.k64, bt.v64 = [None], [None]
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    k, v = (torch.randn((300, 2, D), generator=g, device="cuda").clamp(-3, 3) for _ in range(2))
    store(bt, 0, (k.double() * 2.0 ** k_e).to(bt.dt), v.to(bt.dt))
    bt.q = (bt.q.double().clamp(-3, 3) * 2.0 ** q_e).to(bt.dt)
    got, lse = q.qmm_kv4_attn(bt.q, *bt.args(), ql[0], 300, scale=2.0 ** scale_e, return_lse=True)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    # (the reference's scale is D^-0.5)
    bt.q = bt.q.double() * 2.0 ** scale_e * D ** 0.5
    ref, tol, ls, ltol = reference(bt, True)
    assert ((got.double() - ref).abs() <= tol).all() and ((lse.double() - ls).abs() <= ltol).all()


# A row that sees one key gives its value: the largest weight is rounded to nothing else than itself.
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql,kl,heads,window", [([1], [1], (8, 2), 0), ([1, 2], [500, 40], (8, 2), 1), ([4], [2000], (4, 1), 1),
                                                ([400], [700], (8, 1), 1)])
def test_one_key_gives_its_value(q, dtype, D, ql, kl, heads, window):
    bt = Batch4(ql, kl, *heads, D, dtype)
    out = q.qmm_kv4_attn(bt.q, *bt.args(), max(ql), max(kl), window=window)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    want = torch.cat([v[n - m:] for v, m, n in zip(bt.v64, ql, kl)]).repeat_interleave(heads[0] // heads[1], 1)
    assert torch.equal(out.double(), want)


# Where keys are converted once, max_kv bounds them: a longer sequence counts as one of so many, in whole tiles of 128.
def test_longer_than_max_kv_counts_as_max_kv(q):
    bt = Batch4([1100, 3], [2500, 40], 64, 8, 128, "bf16")
    assert q.qmm_kv4_attn_more_workspace(2, 1103, 64, 8, 128, 1100, 2300) > 0
    got = q.qmm_kv4_attn(bt.q, *bt.args(), 1100, 2300)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 10
    bt.kv_len[0] = 2304
    want = q.qmm_kv4_attn(bt.q, *bt.args(), 1100, 2304)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0 and torch.equal(got, want)
