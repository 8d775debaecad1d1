"""qmm_paged_attn and qmm_kv_append where lengths, masks, scores and arguments are at
their limits: against the plain 64-bit form within its derived bounds
(tests/paged_ref.py), and refusals."""
import math

import pytest
import torch

from paged_ref import Batch, attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_weight_quantized_gb300 as q
    q.load()
    return q


@pytest.fixture(params=["extension", "ctypes"])
def route(q, request, monkeypatch):
    """Either route of the binding to the library."""
    if request.param == "ctypes":
        monkeypatch.setattr(q, "_fast_append", None)
        monkeypatch.setattr(q, "_fast_attn", None)
    elif q._fast_attn is None:
        pytest.skip("extension not built")


def attend(q, bt, window=0, causal=True, max_q=None, max_kv=None, pad=0):
    """out, lse of one call; `pad` rows of NaN follow the batch's queries, which belong to
    no sequence and whose output must stay as it was."""
    query = bt.q
    if pad:
        query = torch.cat([bt.q, torch.full((pad, bt.hq, bt.D), math.nan, dtype=bt.dt, device=bt.q.device)])
    out = torch.full_like(query, 7.0)
    got, lse = q.qmm_paged_attn(query, *bt.args(), (max(bt.ql) if max_q is None else max_q),
                                max(bt.kl) if max_kv is None else max_kv, causal=causal, window=window,
                                return_lse=True, out=out)
    assert got is out
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    assert (out[bt.T:] == 7.0).all()
    return out[:bt.T], lse[:bt.T]


def check(q, bt, window=0, causal=True, **kw):
    out, lse = attend(q, bt, window, causal, **kw)
    ref, tol, ls, ltol = attention(bt, None, causal, window)
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs out of bounds, first at {bad.nonzero()[0].tolist()}"
    empty = torch.isinf(ls)
    assert torch.equal(lse == -math.inf, empty) and (out[empty] == 0).all()
    assert ((lse.double() - ls).abs()[~empty] <= ltol[~empty]).all()
    return out


# the largest window there is; the tiles hold tokens before position 0, too
@pytest.mark.parametrize("n", [3, 50])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5])
def test_window_of_any_size_beside_padding(q, n, window):
    bt = Batch([n, n + 3, 2 * n], [n // 2, 3, n + 300], 8, 2, 128, "bf16", seed=n)
    check(q, bt, window=window)
    check(q, bt, window=window, pad=4000, max_q=4000)


# any bound on the new tokens will do, up to the largest integer
@pytest.mark.parametrize("max_q", [2 ** 31 - 1, 2 ** 28, 70])
@pytest.mark.parametrize("n", [1, 40])
def test_max_q_of_any_size(q, n, max_q):
    check(q, Batch([n, 1, n], [n + 300, 7, n], 16, 2, 64, "f16", seed=n), max_q=max_q)
    check(q, Batch([n], [n + 2000], 8, 1, 128, "bf16", seed=n), max_q=max_q, max_kv=0)


# The kernel for many rows on batches that the other one would take: rows of padding behind the
# batch's tokens raise the bound on a sequence's tokens.
MANY = dict(pad=8192, max_q=8192)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_rows_kernel_every_length(q, D, dtype):
    kl = [1, 2, 3, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 511, 513]
    check(q, Batch([1] * len(kl), kl, 8, 2, D, dtype, seed=D), **MANY)
    check(q, Batch([3, 1, 20], [3, 9000, 500], 8, 2, D, dtype, seed=D), **MANY)


@pytest.mark.parametrize("page,layout", [(1, "hnd"), (7, "nhd"), (8, "hnd"), (24, "gap"), (64, "nhd"), (128, "hnd"),
                                         (200, "gap")])
@pytest.mark.parametrize("n", [1, 70])
def test_many_rows_kernel_pages_and_layouts(q, page, layout, n):
    check(q, Batch([n, n, n], [n, n + 133, n + 470], 4, 2, 128, "f16", page=page, layout=layout, seed=page), **MANY)


@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (7, 1), (17, 1), (64, 1), (40, 8), (100, 1), (128, 1), (258, 2)])
@pytest.mark.parametrize("n", [1, 4, 50])
def test_many_rows_kernel_head_groups(q, heads, n):
    check(q, Batch([n, n], [n + 77, n + 300], *heads, 64, "bf16", seed=heads[0]), **MANY)


@pytest.mark.parametrize("window", [1, 16, 65, 130, 1000])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_many_rows_kernel_window(q, window, n):
    check(q, Batch([n, n, n], [n, n + 90, n + 700], 8, 4, 128, "bf16", seed=window), window=window, **MANY)


@pytest.mark.parametrize("n", [1, 40])
def test_many_rows_kernel_rows_without_keys(q, n):
    bt = Batch([n, n, 0, n, n], [0, n + 50, 30, n // 2, n], 4, 1, 128, "bf16", seed=n)
    for kw in (dict(), dict(causal=False), dict(window=3)):
        assert (check(q, bt, **kw, **MANY)[:n] == 0).all()


# more items, each longer than a block takes whole, than run at once: the axis is split,
# on the counts around one, two and three rounds of blocks
@pytest.mark.parametrize("D,keys", [(64, 560), (128, 300)])
@pytest.mark.parametrize("batch", [29, 33, 60, 93])
def test_more_long_items_than_blocks(q, D, keys, batch):
    kl = [keys + i * 37 % 200 for i in range(batch)]
    check(q, Batch([1] * batch, kl, 64, 32, D, "bf16" if batch % 2 else "f16", page=32, seed=batch))


# NaN and infinite scores: every row that sees such a key gets NaN, as log sum too; the rows
# before it, and the other sequences, are as without it
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,kv,key", [(1, 40, 20), (1, 3000, 2000), (1, 40000, 77), (30, 400, 380), (200, 900, 800),
                                      (130, 6000, 5950)])
def test_nan_reaches_output_and_log_sum(q, n, kv, key, dtype, bad):
    bt = Batch([n, n], [kv, kv - n // 2], 2, 1, 64, dtype, page=16, seed=kv)
    bt.q[..., 0] = 1.0
    clean = attention(bt)
    bt.k_cache[bt.table[0, key // 16], key % 16, 0, 0] = bad
    for pad in (0, 8192):
        out, lse = attend(q, bt, pad=pad, max_q=max(n, pad))
        pos = torch.arange(kv - n, kv, device="cuda")
        hit = torch.cat([pos >= key, torch.zeros(n, dtype=torch.bool, device="cuda")])
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
        ref, tol, ls, ltol = clean
        assert ((out.double() - ref).abs() <= tol)[~hit].all()
        assert ((lse.double() - ls).abs() <= ltol)[~hit].all()


# max_q = 0 in a batch that has tokens: single tokens are answered, more are reported
def test_max_q_of_zero(q, route):
    bt = Batch([1, 1, 1], [90, 5, 700], 8, 2, 64, seed=5)
    check(q, bt, max_q=0)
    wide = Batch([1, 1], [90, 400], 40, 2, 64, seed=6)      # more rows than the decode kernel's tile
    check(q, wide, max_q=0)
    bt = Batch([9, 1], [90, 5], 4, 2, 64, seed=5)
    q.qmm_paged_attn(bt.q, *bt.args(), 0, 90)
    assert q.qmm_device_status() == 10
    assert q.qmm_device_status() == 0


# numbers past 32 bits are refused, not cut
def test_numbers_past_32_bits_are_refused(q, route):
    bt = Batch([2], [10], 4, 2, 64)
    a = bt.args()
    k = torch.zeros(2, 2, 64, device="cuda", dtype=bt.dt)
    big = 2 ** 32 + 5
    for kw in (dict(window=big), dict(max_kv=big), dict(max_q=big)):
        with pytest.raises(ValueError):
            q.qmm_paged_attn(bt.q, *a, **dict(dict(max_q=2, max_kv=10), **kw))
    many = [t[:1].expand(big, -1, -1, -1) for t in a[:2]]
    with pytest.raises(ValueError):
        q.qmm_paged_attn(bt.q, *many, *a[2:], 2, 10)
    with pytest.raises(ValueError):
        q.qmm_kv_append(k, k, *many, *a[2:])
    with pytest.raises(ValueError):
        q.qmm_paged_attn_workspace(8, 2, 64, big)
    assert q.qmm_device_status() == 0


# no memory for the output is torch's own error, by either route
def test_out_of_memory_is_torchs_error(q, route):
    bt = Batch([1], [10], 8, 2, 128)
    query = bt.q[:1].expand(1 << 16, -1, -1)       # an output of 128 MB
    fused = torch.zeros(1, 2, 128, device="cuda", dtype=bt.dt).expand(1 << 16, -1, -1)
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (32 << 20)) / total)
    try:
        with pytest.raises(torch.cuda.OutOfMemoryError):
            q.qmm_paged_attn(query, *bt.args(), 1, 10)
        with pytest.raises(torch.cuda.OutOfMemoryError):
            q.qmm_kv_append(fused, fused, *bt.args(), q=query)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    check(q, bt)


# a sequence of as many keys as there may be (the table names two pages again and again), of
# which the window leaves the last; one key more is reported
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 40])
def test_longest_sequence(q, n, D):
    most, page, w = 2 ** 31 - 16384, 1 << 20, 300
    g = torch.Generator(device="cuda")
    g.manual_seed(n + D)
    k, v = (torch.randn((2, page, 1, D), generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    table = (torch.arange(2048, dtype=torch.int32, device="cuda") % 2).view(1, -1)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    length = torch.tensor([most], dtype=torch.int32, device="cuda")
    x = torch.randn((n, 4, D), generator=g, device="cuda", dtype=torch.float16)
    j = torch.arange(most - n - w, most, device="cuda")
    kk, vv = (t[(j // page) % 2, j % page, 0].double() for t in (k, v))
    pos = torch.arange(most - n, most, device="cuda")[:, None, None]
    see = (j <= pos) & (j > pos - w)
    s = (torch.einsum("thd,jd->thj", x.double(), kk) * D ** -0.5).masked_fill(~see, -math.inf)
    p = torch.softmax(s, -1)
    ref = p @ vv
    tol = 2.0 ** -11 * ref.abs() + (2.0 ** -11 + 2.0 ** -14) * (p @ vv.abs()) + 1e-7      # as in paged_ref
    padded = torch.cat([x, torch.full((8192, 4, D), math.nan, device="cuda", dtype=x.dtype)])
    for x, max_q, max_kv in ((x, n, most), (x, n, 0), (padded, 8192, most)):
        out = q.qmm_paged_attn(x, k, v, table, cu, length, max_q, max_kv, window=w)
        torch.cuda.synchronize()
        assert q.qmm_device_status() == 0
        assert ((out[:n].double() - ref).abs() <= tol).all()
    q.qmm_kv_append(k[0, :n], v[0, :n], k, v, table, cu, length)
    assert q.qmm_device_status() == 0
    q.qmm_paged_attn(x, k, v, table, cu, length + 1, n, 0, window=w)
    assert q.qmm_device_status() == 10
    q.qmm_kv_append(k[0, :n], v[0, :n], k, v, table, cu, length + 1)
    assert q.qmm_device_status() == 10
    assert q.qmm_device_status() == 0


# lengths below zero, down to the smallest integer: padding, as zero is
@pytest.mark.parametrize("length", [-1, -2 ** 31 + 2, -2 ** 31])
def test_negative_lengths_are_padding(q, length):
    bt = Batch([3, 5], [20, 40], 4, 2, 64, seed=4)
    bt.kv_len[1] = length
    k = torch.ones(8, 2, 64, device="cuda", dtype=bt.dt)
    before, sentinel = bt.k_cache.clone(), torch.full_like(bt.q, 7.0)
    q.qmm_kv_append(k, k, *bt.args(), q=bt.q, q_out=sentinel)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    assert (sentinel[3:] == 7.0).all() and torch.equal(sentinel[:3], bt.q[:3])
    changed = torch.nan_to_num(bt.k_cache.double(), nan=5e5) != torch.nan_to_num(before.double(), nan=5e5)
    assert int(changed.any(-1).sum()) == 6          # 3 slots of 2 heads
    out, lse = q.qmm_paged_attn(bt.q[3:], bt.k_cache, bt.v_cache, bt.table[1:], bt.cu_q[1:] - 3, bt.kv_len[1:], 5, 40,
                                return_lse=True)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    assert (out == 0).all() and (lse == -math.inf).all()


# rows of padding behind the batch may hold anything, and nothing is stored for them
def test_append_leaves_padding_alone(q):
    bt = Batch([2, 3], [20, 30], 4, 2, 64, seed=4)
    fused = torch.full((400, 8, 64), math.nan, device="cuda", dtype=bt.dt)
    fused[:5] = torch.randn(5, 8, 64, device="cuda").to(bt.dt)
    other = Batch([2, 3], [20, 30], 4, 2, 64, seed=4)
    want = q.qmm_kv_append(fused[:5, 4:6], fused[:5, 6:], *other.args(), q=fused[:5, :4])
    out = torch.full((400, 4, 64), 7.0, device="cuda", dtype=bt.dt)
    q.qmm_kv_append(fused[:, 4:6], fused[:, 6:], *bt.args(), q=fused[:, :4], q_out=out)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    assert torch.equal(out[:5], want) and (out[5:] == 7.0).all()
    for a, b in ((bt.k_cache, other.k_cache), (bt.v_cache, other.v_cache)):
        assert torch.equal(torch.nan_to_num(a.double(), nan=9e9), torch.nan_to_num(b.double(), nan=9e9))


# a table without columns holds no keys
@pytest.mark.parametrize("n", [1, 40, 600])
def test_empty_table(q, n):
    bt = Batch([n], [0], 16, 2, 64, seed=4)
    none = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    for window in (0, 5):
        out = q.qmm_paged_attn(bt.q, bt.k_cache, bt.v_cache, none, bt.cu_q, bt.kv_len, n, 0, window=window)
        torch.cuda.synchronize()
        assert (out == 0).all() and q.qmm_device_status() == 0
    q.qmm_paged_attn(bt.q, bt.k_cache, bt.v_cache, none, bt.cu_q, bt.kv_len + 1, n, 0)
    assert q.qmm_device_status() == 10
