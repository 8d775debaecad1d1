"""qmm_kv4_append, qmm_kv4_read and qmm_kv4_attn against plain 64-bit forms
(tests/kv4_ref.py): the codes and scales bit for bit, attention within derived bounds."""
import math

import pytest
import torch

from kv4_ref import Batch4, attention4, normed, pack, patterns, positions, quantize, rotate, values
from paged_ref import TYPES, U, cos_sin_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_weight_quantized_gb300 as q
    q.load()
    return q


def status(q):
    torch.cuda.synchronize()
    return q.qmm_device_status()


# ---- attention -----------------------------------------------------------------
def check(q, bt, window=0, sinks=0, causal=True, max_q=None, max_kv=None, pad=0, scale=None):
    query = bt.q
    if pad:
        query = torch.cat([bt.q, torch.full((pad, bt.hq, bt.D), math.nan, dtype=bt.dt, device=bt.q.device)])
    out = torch.full_like(query, 7.0)
    got, lse = q.qmm_kv4_attn(query, *bt.args(), (max(bt.ql) if max_q is None else max_q),
                              max(bt.kl) if max_kv is None else max_kv, scale=scale, causal=causal, window=window,
                              sinks=sinks, return_lse=True, out=out)
    assert got is out
    assert status(q) == 0
    assert (out[bt.T:] == 7.0).all()
    out, lse = out[:bt.T], lse[:bt.T]
    ref, tol, ls, ltol = attention4(bt, scale, causal, window, sinks)
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs out of bounds, first at {bad.nonzero()[0].tolist()}"
    empty = torch.isinf(ls)
    assert torch.equal(lse == -math.inf, empty) and (out[empty] == 0).all()
    assert ((lse.double() - ls).abs()[~empty] <= ltol[~empty]).all()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 8, 16])
@pytest.mark.parametrize("kl", [[1], [17, 1, 40], [517], [2, 130, 1000, 31]])
def test_single_tokens(q, dtype, D, group, kl):
    check(q, Batch4([1] * len(kl), kl, 2 * group, 2, D, dtype, seed=group))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "gaps"])
@pytest.mark.parametrize("page", [1, 7, 16, 48, 128])
def test_layouts_and_pages(q, dtype, layout, page):
    check(q, Batch4([1, 3], [100, 333], 6, 3, 128 if page != 48 else 64, dtype, page=page, layout=layout, seed=page))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql,kl", [([5, 2, 7], [600, 40, 7]), ([1, 40, 0, 9], [300, 40, 12, 2000]),
                                   ([130], [130]), ([300, 1, 17], [1000, 700, 17]), ([129, 64], [129, 1024])])
@pytest.mark.parametrize("causal", [True, False])
def test_several_tokens(q, D, ql, kl, causal):
    check(q, Batch4(ql, kl, 8, 2, D, "bf16", seed=len(ql)), causal=causal)
    check(q, Batch4(ql, kl, 7, 1, D, "f16", page=8, seed=3), causal=causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 33, 200, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 4, 150, 2 ** 31 - 1])
@pytest.mark.parametrize("ql", [[1, 1, 1], [3, 40, 200]])
def test_windows_and_first_tokens(q, D, window, sinks, ql):
    bt = Batch4(ql, [2000, 641, 260], 8, 2, D, "f16" if sinks % 2 else "bf16", seed=window % 100)
    check(q, bt, window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("batch,n", [(1, 30000), (3, 9000), (40, 1500)])
def test_split_axes(q, D, batch, n):
    bt = Batch4([1] * batch, [max(1, n - 700 * (i % 5)) for i in range(batch)], 8, 2, D, "bf16", page=64)
    a = check(q, bt)
    assert torch.equal(a, check(q, bt))               # the same run to run
    check(q, bt, max_kv=0)
    check(q, bt, max_kv=2 ** 31 - 1, max_q=2 ** 31 - 1)


# Long prompts: keys converted once in the workspace, against converted by every block, and
# against the plain form.
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,heads,ql,kl,page,layout", [
    (128, (64, 8), [1030], [2100], 16, "hnd"), (64, (32, 4), [600, 3, 0, 1030], [900, 3, 5, 3000], 7, "nhd"),
    (128, (24, 8), [1300, 1200], [1641, 5000], 48, "gaps")])
@pytest.mark.parametrize("window,causal", [(0, True), (0, False), (2700, True)])
def test_keys_converted_once(q, dtype, D, heads, ql, kl, page, layout, window, causal):
    bt = Batch4(ql, kl, *heads, D, dtype, page=page, layout=layout)
    more = q.qmm_kv4_attn_more_workspace(len(ql), sum(ql), *heads, D, max(ql), max(kl))
    assert more >= 4 * len(ql) * max(kl) * heads[1] * D
    a = check(q, bt, window=window, causal=causal)
    ws = torch.empty(q.qmm_kv4_attn_workspace(*heads, D, max(ql)), dtype=torch.uint8, device="cuda")
    b = q.qmm_kv4_attn(bt.q, *bt.args(), max(ql), max(kl), window=window, causal=causal, workspace=ws)
    assert status(q) == 0
    if not window:
        assert torch.equal(a, b)
    ref, tol, _, _ = attention4(bt, None, causal, window)
    assert ((b.double() - ref).abs() <= tol).all()
    # a workspace of the caller's, aligned to less than the converted keys need
    full = torch.empty(ws.numel() + more + 16, dtype=torch.uint8, device="cuda")
    for at in (0, 16):
        full.fill_(255)
        c = q.qmm_kv4_attn(bt.q, *bt.args(), max(ql), max(kl), window=window, causal=causal, workspace=full[at:])
        assert status(q) == 0 and torch.equal(c, a if at == 0 else b)


# Captured: every replay converts the keys that lie in the cache then, for two calls that share
# their workspace and on another stream than the capture's.
def test_converted_keys_in_a_graph(q):
    bt, other = Batch4([1030], [2100], 64, 8, 128, "bf16"), Batch4([1030], [2100], 64, 8, 128, "bf16", seed=5)
    more = q.qmm_kv4_attn_more_workspace(1, 1030, 64, 8, 128, 1030, 2100)
    ws = torch.empty(q.qmm_kv4_attn_workspace(64, 8, 128, 1030) + more, dtype=torch.uint8, device="cuda")
    run = lambda b: q.qmm_kv4_attn(b.q, *b.args(), 1030, 2100, workspace=ws)
    want = [run(b) for b in (bt, other)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [run(b) for b in (bt, other)]
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for a, b in ((bt.k_cache, other.k_cache), (bt.v_cache, other.v_cache), (bt.scales, other.scales), (bt.q, other.q),
                 (bt.table, other.table)):
        a.copy_(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    side.synchronize()
    assert status(q) == 0 and torch.equal(got[0], want[1]) and torch.equal(got[1], want[1])


# A prompt beside sequences of a token: its keys alone would be worth it.
def test_keys_of_mixed_batches_stay(q):
    assert q.qmm_kv4_attn_more_workspace(1, 2048, 64, 8, 128, 2048, 8192) > 0
    assert q.qmm_kv4_attn_more_workspace(16, 2048 + 15, 64, 8, 128, 2048, 8192) == 0


# Where memory is short, a call does without the scratch for converted keys.
@pytest.mark.parametrize("fast", [True, False])
def test_converted_keys_without_memory(q, fast, monkeypatch):
    if not fast:
        monkeypatch.setattr(q, "_fast_kv4_attn", None)
    bt = Batch4([1030], [8000], 64, 8, 128, "bf16")
    want = q.qmm_kv4_attn(bt.q, *bt.args(), 1030, 8000)
    more = q.qmm_kv4_attn_more_workspace(1, 1030, 64, 8, 128, 1030, 8000)
    base = q.qmm_kv4_attn_workspace(64, 8, 128, 1030)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    try:
        room = torch.cuda.memory_reserved() + want.nbytes + base + more // 2
        torch.cuda.set_per_process_memory_fraction(room / total)
        got = q.qmm_kv4_attn(bt.q, *bt.args(), 1030, 8000)
        with pytest.raises(torch.OutOfMemoryError):
            torch.empty(base + more, dtype=torch.uint8, device="cuda")
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert status(q) == 0 and torch.equal(got, want)


def test_longer_than_max_kv_is_recorded(q):
    bt = Batch4([1100], [2500], 64, 8, 128, "bf16")
    assert q.qmm_kv4_attn_more_workspace(1, 1100, 64, 8, 128, 1100, 1920) > 0
    q.qmm_kv4_attn(bt.q, *bt.args(), 1100, 4000)
    assert status(q) == 0
    # than the table
    ws = torch.empty(q.qmm_kv4_attn_workspace(64, 8, 128, 1100) +
                     q.qmm_kv4_attn_more_workspace(1, 1100, 64, 8, 128, 1100, 2500), dtype=torch.uint8, device="cuda")
    run = lambda table: q.qmm_kv4_attn(bt.q, *bt.args()[:3], table, *bt.args()[4:], 1100, 2500, workspace=ws.fill_(255))
    short = run(bt.table[:, :120].contiguous())
    assert status(q) == 10 and torch.isfinite(short).all()
    # pages that are not there: keys and values of zeros
    bad = bt.table.clone()
    bad[0, 3] = -1
    bad[0, 7] = bt.k_cache.shape[0]
    got = run(bad)
    assert status(q) == 10
    direct = q.qmm_kv4_attn(bt.q, *bt.args()[:3], bad, *bt.args()[4:], 1100, 2500, workspace=ws[:-4096])
    assert status(q) == 10 and torch.equal(got, direct)
    # than max_kv
    assert q.qmm_kv4_attn_more_workspace(1, 1100, 64, 8, 128, 1100, 2300) > 0
    q.qmm_kv4_attn(bt.q, *bt.args(), 1100, 2300)
    assert status(q) == 10


def test_padding(q):
    bt = Batch4([1, 0, 2, 1], [0, 5, 1, 50], 8, 2, 128, "bf16", extra_blocks=3)
    check(q, bt, pad=5)
    check(q, bt, window=3, sinks=1, pad=1)


def test_nan_and_infinite_queries(q):
    bt = Batch4([1, 1, 2], [40, 70, 90], 8, 2, 128, "bf16")
    bt.q[1, 3, 7] = math.nan
    bt.q[2, 0, 100] = math.inf
    out, lse = q.qmm_kv4_attn(bt.q, *bt.args(), 2, 90, return_lse=True)
    assert status(q) == 0
    bad = torch.zeros_like(lse, dtype=torch.bool)
    bad[1, 3] = bad[2, 0] = True
    assert torch.equal(lse.isnan(), bad) and torch.equal(out.isnan().any(-1), bad) and torch.equal(out.isnan().all(-1), bad)


# queries far from one and values whose scales grow and shrink along the axis
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [1e-4, 300.0])
def test_magnitudes(q, dtype, size):
    bt = Batch4([1, 4], [700, 333], 8, 2, 128, dtype, spread=1.0)
    bt.q = (bt.q.float() * size).to(bt.dt)
    check(q, bt, scale=bt.D ** -0.5 / size)


def test_strides_of_queries(q):
    bt = Batch4([1, 3], [100, 50], 8, 2, 128, "bf16")
    wide = torch.zeros(bt.T, 8 + 4, 128, dtype=bt.dt, device="cuda")
    wide[:, :8] = bt.q
    ref = check(q, bt)
    assert torch.equal(q.qmm_kv4_attn(wide[:, :8], *bt.args(), 3, 100), ref)


def test_graph_replays_on_new_lengths(q):
    bt = Batch4([1, 1], [300, 200], 8, 2, 128, "bf16")
    ws = torch.empty(q.qmm_kv4_attn_workspace(8, 2, 128, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(bt.q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        q.qmm_kv4_attn(bt.q, *bt.args(), 1, 300, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qmm_kv4_attn(bt.q, *bt.args(), 1, 300, out=out, workspace=ws)
    for kl in ([300, 200], [150, 7]):
        bt.kv_len.copy_(torch.tensor(kl, dtype=torch.int32))
        bt.kl, old = kl, (bt.k64, bt.v64)
        bt.k64, bt.v64 = [x[:n] for x, n in zip(old[0], kl)], [x[:n] for x, n in zip(old[1], kl)]
        graph.replay()
        torch.cuda.synchronize()
        ref, tol, _, _ = attention4(bt)
        bt.k64, bt.v64 = old
        assert ((out.double() - ref).abs() <= tol).all()
    assert q.qmm_device_status() == 0


def test_bad_pages_and_lengths_are_recorded(q):
    bt = Batch4([1], [100], 8, 2, 128, "bf16")
    bt.table[0, 2] = 10 ** 6
    q.qmm_kv4_attn(bt.q, *bt.args(), 1, 100)
    assert status(q) == 10
    q.qmm_kv4_read(*bt.args(), 1)                      # (the last key lies in a good page)
    assert status(q) == 0
    bt.kv_len.fill_(10 ** 7)
    q.qmm_kv4_read(*bt.args(), 1)
    assert status(q) == 10
    q.qmm_kv4_attn(bt.q, *bt.args(), 1, 100)
    assert status(q) == 10


# ---- append and read --------------------------------------------------------------
def append(q, bt, rot, interleaved, norm, seed=0, with_q=True):
    """One append of random rows into an empty cache: the rows, what came out."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = torch.randn((bt.T, bt.hq + 2 * bt.hk, bt.D), generator=g, device="cuda").to(bt.dt)
    qkv *= torch.exp2(torch.randint(-3, 4, (bt.T, 1, 1), generator=g, device="cuda")).to(bt.dt)
    x, k, v = qkv[:, :bt.hq], qkv[:, bt.hq:bt.hq + bt.hk], qkv[:, bt.hq + bt.hk:]
    cs = cos_sin_table(max(bt.kl), rot) if rot else None
    w = [(1 + torch.randn(bt.D, generator=g, device="cuda") / 4).to(bt.dt) if n else None for n in norm]
    got = q.qmm_kv4_append(k, v, *bt.args(), q=x if with_q else None, cos_sin=cs, interleaved=interleaved,
                           q_norm=w[0] if with_q else None, k_norm=w[1], eps=1e-5)
    assert status(q) == 0
    return x, k, v, cs, w, got


def stored(bt):
    """Codes and patterns of the batch's tokens, as they lie in the cache."""
    seq, pos = positions(bt)
    page = bt.table.long()[seq, pos // bt.page]
    s = bt.scales.view(torch.int16)[page, pos % bt.page].view(bt.dt)
    half = bt.D // 64
    return (bt.k_cache[page, pos % bt.page], s[..., :half].contiguous()), (bt.v_cache[page, pos % bt.page], s[..., half:].contiguous())


CASES = [([3], [3]), ([1, 1, 1], [1, 17, 400]), ([33, 0, 5], [40, 12, 5])]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql,kl", CASES)
@pytest.mark.parametrize("rot,interleaved", [(0, False), (32, False), (48, True), (64, False), (64, True), (128, False), (128, True)])
def test_append_stores_the_plain_codes(q, dtype, D, ql, kl, rot, interleaved):
    """Without norms every step is the same in any IEEE arithmetic: bit for bit."""
    if rot > D:
        pytest.skip("rotation wider than the head")
    bt = Batch4(ql, kl, 6, 3, D, dtype, page=16 if rot else 7, layout="nhd" if rot == 32 else "hnd", fill=False)
    before = [t.clone() for t in (bt.k_cache, bt.v_cache, bt.scales.view(torch.int16))]
    x, k, v, cs, _, got = append(q, bt, rot, interleaved, (False, False), seed=rot)
    seq, pos = positions(bt)

    def turned(y):     # in fp32, product by product
        y = y.float()
        if not rot:
            return y
        c, s = cs[pos, :rot // 2][:, None], cs[pos, rot // 2:][:, None]
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
        a, b = a * c - b * s, b * c + a * s
        return torch.cat([torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1), y[..., rot:]], -1)

    assert torch.equal(got, turned(x).to(bt.dt))
    for (codes, pats), y in zip(stored(bt), (turned(k).to(bt.dt), v)):
        c, s, z = quantize(y)
        assert torch.equal(pats.view(torch.int16), patterns(s, z, bt.dt).view(torch.int16))
        assert torch.equal(codes, pack(c))
    # and nothing else
    page = bt.table.long()[seq, pos // bt.page]
    for was, now in zip(before, (bt.k_cache, bt.v_cache, bt.scales.view(torch.int16))):
        now = now.clone()
        now[page, pos % bt.page] = was[page, pos % bt.page]
        assert torch.equal(was, now)
    # what reading gives is exact
    kr, vr = q.qmm_kv4_read(*bt.args(), bt.T)
    for y, (codes, pats) in zip((kr, vr), stored(bt)):
        assert torch.equal(y.double(), values(codes, pats))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("norm", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("rot,interleaved,heads", [(0, False, (5, 1)), (64, False, (6, 3)), (64, True, (1, 1)), (32, False, (24, 8))])
def test_append_with_norms(q, dtype, D, norm, rot, interleaved, heads):
    bt = Batch4([40, 1], [60, 333], *heads, D, dtype, fill=False)
    x, k, v, cs, w, got = append(q, bt, rot, interleaved, norm, seed=D)
    _, pos = positions(bt)
    u = U[bt.dt]
    # the sum of D squares is off by D 2^-24 at most, half of that goes to its root; eight
    # more roundings; a rotated value is below |a| + |b|, 2 max |x|
    err = (D / 2 + 8) * 2.0 ** -24
    ref = rotate(normed(x, w[0], 1e-5), pos, cs, interleaved)
    big = ref.abs().amax(-1, keepdim=True)
    assert ((got.double() - ref).abs() <= u * ref.abs() + 2 * err * big + 1e-12).all()
    ref = rotate(normed(k, w[1], 1e-5), pos, cs, interleaved)
    (codes, pats), (vcodes, vpats) = stored(bt)
    off = u * ref.abs() + 2 * err * ref.abs().amax(-1, keepdim=True) + 1e-12
    s = ((pats.view(torch.int16) & -16).view(bt.dt).double())[..., None].expand(-1, -1, -1, 64).flatten(-2)
    assert ((values(codes, pats) - ref).abs() <= s / 2 + off).all()
    # the scales are the smallest that will do, or one of their steps from it
    want = quantize(ref.to(bt.dt))[1]
    assert ((s[..., ::64] - want).abs() <= want * 2.0 ** (1 - (4 if dtype == "bf16" else 7))).all()
    c, s, z = quantize(v)
    assert torch.equal(vcodes, pack(c)) and torch.equal(vpats.view(torch.int16), patterns(s, z, bt.dt).view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_of_odd_groups(q, dtype, D):
    """Zeros, one sign, one value, the smallest and the largest numbers, and NaN."""
    dt = TYPES[dtype]
    bt = Batch4([8], [8], 2, 1, D, dtype, fill=False)
    f = torch.finfo(dt)
    tiny = f.smallest_normal
    v = torch.zeros(8, 1, D, dtype=dt, device="cuda")
    v[1] = 3.0
    v[2] = -0.37
    v[3, 0, 5] = f.max
    v[3, 0, 9] = -f.max
    v[4, 0] = torch.linspace(-1, 1, D, device="cuda").to(dt) * tiny
    v[5, 0] = torch.linspace(f.max / 2, f.max, D, device="cuda", dtype=torch.float64).to(dt)
    v[6, 0, 3] = f.smallest_normal * f.eps                        # the smallest number
    v[7] = torch.randn(1, D, device="cuda").to(dt)
    q.qmm_kv4_append(v, v, *bt.args())
    kr, vr = q.qmm_kv4_read(*bt.args(), 8)
    assert status(q) == 0
    assert torch.equal(kr, vr) and vr.isfinite().all()
    c, s, z = quantize(v)
    assert torch.equal(stored(bt)[1][0], pack(c))
    assert torch.equal(vr.double(), values(pack(c), patterns(s, z, dt)))
    for bad in (math.nan, math.inf, -math.inf):
        v[7, 0, 2] = bad
        q.qmm_kv4_append(v, v, *bt.args())
        vr = q.qmm_kv4_read(*bt.args(), 8)[1]
        assert status(q) == 0
        assert vr[7, 0, :64].isnan().all() and vr[7, 0, 64:].isfinite().all() and vr[:7].isfinite().all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "gaps"])
@pytest.mark.parametrize("ql,kl,page,hk", [([1], [1], 16, 1), ([100, 0, 7], [100, 9, 400], 24, 3), ([5000], [5000], 64, 2), ([1, 1], [9, 8], 1, 5)])
def test_read(q, D, layout, ql, kl, page, hk):
    bt = Batch4(ql, kl, hk, hk, D, "bf16", page=page, layout=layout)
    k = torch.full((bt.T + 3, hk, D), 7.0, dtype=bt.dt, device="cuda")
    v = k.clone()
    a, b = q.qmm_kv4_read(*bt.args(), bt.T + 3, k_out=k, v_out=v)
    assert a is k and b is v and status(q) == 0
    assert torch.equal(k[:bt.T].double(), torch.cat([x[n - m:] for x, m, n in zip(bt.k64, ql, kl)]))
    assert torch.equal(v[:bt.T].double(), torch.cat([x[n - m:] for x, m, n in zip(bt.v64, ql, kl)]))
    assert (k[bt.T:] == 7.0).all() and (v[bt.T:] == 7.0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_read_into_rows_aligned_to_16_bytes(q, D):
    bt = Batch4([5], [40], 3, 3, D, "f16")
    a, b = (torch.full((5 * 3 * D + 16,), 7.0, dtype=bt.dt, device="cuda") for _ in range(2))
    k, v = a[8:8 + 5 * 3 * D].view(5, 3, D), b[8:8 + 5 * 3 * D].view(5, 3, D)
    q.qmm_kv4_read(*bt.args(), 5, k_out=k, v_out=v)
    assert status(q) == 0
    assert torch.equal(k.double(), bt.k64[0][35:]) and torch.equal(v.double(), bt.v64[0][35:])
    for x in (a, b):
        assert (x[:8] == 7.0).all() and (x[-8:] == 7.0).all()


def test_padding_is_left_alone(q):
    bt = Batch4([1, 2, 1], [0, 1, 3], 4, 2, 128, "bf16", fill=False, extra_blocks=1)
    g = torch.randn(bt.T + 2, 8, 128, device="cuda").bfloat16()
    out = torch.full((bt.T + 2, 4, 128), 7.0, dtype=bt.dt, device="cuda")
    q.qmm_kv4_append(g[:, 4:6], g[:, 6:], *bt.args(), q=g[:, :4], q_out=out)
    assert status(q) == 0
    kept = torch.tensor([True, True, False, False, True, True], device="cuda")   # tokens without a position, past the batch
    assert (out[kept] == 7.0).all() and torch.equal(out[~kept], g[:, :4][~kept])
    k = torch.full((bt.T + 2, 2, 128), 7.0, dtype=bt.dt, device="cuda")
    q.qmm_kv4_read(*bt.args(), bt.T + 2, k_out=k)
    assert status(q) == 0
    assert (k[kept] == 7.0).all() and k[~kept].isfinite().all()


def test_queries_in_place_and_without(q):
    bt = Batch4([7], [20], 4, 2, 128, "f16", fill=False)
    x, k, v, cs, w, got = append(q, bt, 64, False, (True, True))
    first = [t.clone() for t in (bt.k_cache, bt.v_cache, bt.scales.view(torch.int16))]
    y = x.contiguous().clone()
    assert q.qmm_kv4_append(k, v, *bt.args(), q=y, q_out=y, cos_sin=cs, q_norm=w[0], k_norm=w[1], eps=1e-5) is y
    assert torch.equal(y, got)
    assert q.qmm_kv4_append(k, v, *bt.args(), cos_sin=cs, k_norm=w[1], eps=1e-5) is None
    assert status(q) == 0
    for a, b in zip(first, (bt.k_cache, bt.v_cache, bt.scales.view(torch.int16))):
        assert torch.equal(a, b)


# ---- a decoder's use of them together ------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_prompt_and_steps(q, dtype):
    """A prompt in two chunks, then single tokens, every one attending to what was stored:
    against dense attention over the values that reading back gives."""
    D, hq, hk, page, n = 128, 8, 2, 16, 75
    dt = TYPES[dtype]
    bt = Batch4([n], [n], hq, hk, D, dtype, page=page, fill=False)
    x = torch.randn(n, hq + 2 * hk, D, device="cuda").to(dt)
    cs = cos_sin_table(n, D)
    wq, wk = (1 + torch.randn(2, D, device="cuda") / 4).to(dt)
    outs, turned, at = [], [], 0
    for m in (40, 30, 1, 1, 2, 1):
        rows = x[at:at + m]
        cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        length = torch.tensor([at + m], dtype=torch.int32, device="cuda")
        cache = bt.k_cache, bt.v_cache, bt.scales, bt.table, cu, length
        y = q.qmm_kv4_append(rows[:, hq:hq + hk], rows[:, hq + hk:], *cache, q=rows[:, :hq], cos_sin=cs, q_norm=wq, k_norm=wk)
        outs.append(q.qmm_kv4_attn(y, *cache, m, at + m, window=20, sinks=3))
        turned.append(y)
        at += m
    k, v = q.qmm_kv4_read(*bt.args(), n)
    assert status(q) == 0
    bt.q, bt.k64, bt.v64 = torch.cat(turned), [k.double()], [v.double()]
    ref, tol, _, _ = attention4(bt, window=20, sinks=3)
    assert ((torch.cat(outs).double() - ref).abs() <= tol).all()
    # and what was stored is the rows: within a step's half and a rounding of the type
    ref = rotate(normed(x[:, hq:hq + hk], wk, 1e-6), torch.arange(n, device="cuda"), cs, False)
    near = ref.unflatten(-1, (-1, 64)).abs().amax(-1, keepdim=True)
    assert ((k.double() - ref).unflatten(-1, (-1, 64)).abs() <= near * (2 / 15 * (1 + 2.0 ** -3) / 2 + 2 * U[dt])).all()
