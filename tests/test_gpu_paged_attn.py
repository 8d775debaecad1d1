"""GPU parity of qmm_paged_attn against the plain 64-bit form, element by element
within bounds derived from the roundings (tests/paged_ref.py), over lengths,
pages, layouts, head groups, masks and splits."""
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
        monkeypatch.setattr(q, "_fast_attn", None)
    elif q._fast_attn is None:
        pytest.skip("extension not built")


def check(q, bt, scale=None, causal=True, window=0, max_kv=None, max_q=None, query=None):
    """One call, and where the lengths leave the choice, one with a max_q so large that the
    chunk kernel runs: both against the plain form."""
    if max_q is None and max(bt.ql) > 1:
        check(q, bt, scale, causal, window, max_kv, 4096, query)
    out, lse = q.qmm_paged_attn(bt.q if query is None else query, *bt.args(),
                                max(bt.ql) if max_q is None else max_q, max(bt.kl) if max_kv is None else max_kv,
                                scale=scale, causal=causal, window=window, return_lse=True)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    ref, tol, ls, ltol = attention(bt, scale, causal, window)
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs out of bounds, first at {bad.nonzero()[0].tolist()}"
    empty = torch.isinf(ls)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    assert (out[empty] == 0).all()
    d = (lse.double() - ls).abs()
    assert (d[~empty] <= ltol[~empty]).all(), float((d - ltol)[~empty].max())
    return out


# single tokens: every length around the kernels' tiles (16, 64, 128 keys)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_single_tokens_every_length(q, D, dtype):
    kl = [1, 2, 3, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 511, 513]
    check(q, Batch([1] * len(kl), kl, 8, 2, D, dtype, seed=D))


# chunks of every length, also of a length near or equal to the keys'
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_chunks_every_length(q, D, dtype):
    ql = [1, 2, 5, 31, 32, 33, 64, 65, 127, 128, 129, 200, 3, 260]
    kl = [1, 2, 300, 31, 40, 129, 64, 128, 127, 257, 1000, 200, 515, 261]
    check(q, Batch(ql, kl, 8, 2, D, dtype, seed=D + 1))


@pytest.mark.parametrize("page,layout", [(1, "hnd"), (7, "nhd"), (8, "hnd"), (24, "gap"), (64, "nhd"), (128, "hnd"),
                                         (200, "gap")])
@pytest.mark.parametrize("n", [1, 70])
def test_pages_and_layouts(q, page, layout, n):
    check(q, Batch([n, n, n], [n, n + 133, n + 470], 4, 2, 128, "f16", page=page, layout=layout, seed=page))


@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (6, 2), (7, 1), (16, 1), (17, 1), (64, 1), (40, 8), (32, 32), (100, 1), (128, 1), (258, 2)])
@pytest.mark.parametrize("n", [1, 4, 50])
def test_head_groups(q, heads, n):
    check(q, Batch([n, n], [n + 77, n + 300], *heads, 64, "bf16", seed=heads[0]))


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 130, 1000])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_window(q, window, n):
    check(q, Batch([n, n, n], [n, n + 90, n + 700], 8, 4, 128, "bf16", seed=window), window=window)


@pytest.mark.parametrize("n", [1, 20, 140])
def test_not_causal(q, n):
    check(q, Batch([n, n], [n + 5, n + 400], 8, 2, 64, "f16", seed=n), causal=False)


# rows whose mask leaves nothing: sequences without keys, tokens before position 0,
# sequences without new tokens
@pytest.mark.parametrize("n", [1, 40])
def test_rows_without_keys(q, n):
    bt = Batch([n, n, 0, n, n], [0, n + 50, 30, n // 2, n], 4, 1, 128, "bf16", seed=n)
    out = check(q, bt)
    assert (out[:n] == 0).all()
    check(q, bt, causal=False)
    check(q, bt, window=3)


def test_no_tokens(q, route):
    bt = Batch([0, 0], [5, 9], 4, 2, 64)
    assert q.qmm_paged_attn(bt.q, *bt.args(), 1, 9).shape == (0, 4, 64)
    assert q.qmm_device_status() == 0


# one long sequence is split over every block and joined
@pytest.mark.parametrize("n,kv", [(1, 40001), (4, 20000), (33, 30011), (200, 9999)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_axis_is_split(q, n, kv, dtype):
    check(q, Batch([n], [kv], 8, 2, 128, dtype, page=64, seed=kv))


# short axes: clusters of two to eight blocks of eight and of four warps, single blocks of
# both, and axes that are split, by the number of sequences and of keys
@pytest.mark.parametrize("batch", [1, 5, 13, 30, 70, 160])
@pytest.mark.parametrize("D", [64, 128])
def test_short_axes(q, batch, D):
    for kv in (40, 190, 450, 1100, 2300, 4500):
        if batch * kv <= 160000:
            check(q, Batch([1] * batch, [max(1, kv - i % 3 * 31) for i in range(batch)], 8, 2, D, "bf16", seed=kv))


# several items a block, of which the second 128 rows' warps have a part in few: a wide one
# and then more one-tile items of at most 128 rows than are found ahead
@pytest.mark.parametrize("D", [64, 128])
def test_wide_items_between_narrow_ones(q, D):
    ql = [200 if i % 3 == 0 else 90 + i % 39 for i in range(120)]
    check(q, Batch(ql, ql, 8, 8, D, "f16", seed=7))


# more short items than run at once, some without keys, some with a window
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("most", [5, 100, 250])
def test_many_short_items(q, D, most):
    kl = [i * 7 % (most + 1) for i in range(150)]
    check(q, Batch([1] * 150, kl, 16, 8, D, "f16", seed=most))
    check(q, Batch([1] * 150, [900 + k for k in kl], 16, 8, D, "bf16", seed=most + 1), window=most)


# ragged batches: long and short items on the same blocks
@pytest.mark.parametrize("n", [1, 48])
def test_ragged(q, n):
    kl = [n + (i * i * 37) % 3001 for i in range(40)]
    check(q, Batch([n] * 40, kl, 4, 2, 64, "f16", seed=3), window=0)
    check(q, Batch([n] * 40, kl, 4, 2, 64, "f16", seed=4), window=100)


# the running maximum grows along the keys: the output is rescaled again and again,
# by small and by huge factors; scores far apart
@pytest.mark.parametrize("n", [1, 130])
@pytest.mark.parametrize("step", [0.02, 0.5])
def test_growing_maximum(q, n, step):
    bt = Batch([n, n], [n + 700, n + 1500], 4, 2, 128, "bf16", seed=9)
    bt.q[:] = 0
    bt.q[..., 0] = 16.0
    for b in range(2):
        kv = bt.kl[b]
        ramp = (torch.arange(kv, device="cuda", dtype=torch.float32) * step).to(bt.dt)
        bt.k64[b][..., 0] = ramp.double()[:, None]
        for i in range(-(-kv // bt.page)):
            m = min(bt.page, kv - i * bt.page)
            bt.k_cache[bt.table[b, i], :m, :, 0] = ramp[i * bt.page:i * bt.page + m, None]
    check(q, bt)


# a scale that makes a few keys take everything, and one that flattens the weights
@pytest.mark.parametrize("scale", [2.0, 1e-3])
@pytest.mark.parametrize("n", [1, 60])
def test_scales(q, scale, n):
    check(q, Batch([n], [n + 900], 4, 2, 64, "f16", seed=5, spread=0.3 if scale > 1 else 1.0), scale=scale)


# keys that nobody may read hold infinities and NaN (Batch fills unused slots with
# NaN already); here slots before the window, whose pages are gone from the table
@pytest.mark.parametrize("n", [1, 30])
def test_pages_before_the_window_are_not_read(q, n):
    w, kv = 50, n + 1000
    bt = Batch([n], [kv], 4, 1, 128, "bf16", seed=2)
    ref, tol, _, _ = attention(bt, window=w)
    first = kv - n - w + 1
    bt.table[0, :first // bt.page] = -1
    for i in range(first % bt.page):
        slot = first // bt.page
        bt.k_cache[bt.table[0, slot], i] = float("inf")
        bt.v_cache[bt.table[0, slot], i] = float("nan")
    out = q.qmm_paged_attn(bt.q, *bt.args(), n, kv, window=w)
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    assert ((out.double() - ref).abs() <= tol).all()


def test_infinite_and_nan_scores_propagate(q):
    bt = Batch([1, 1], [40, 40], 1, 1, 64, "f16", seed=1)
    bt.k_cache[bt.table[0, 1], 3] = float("nan")
    out = q.qmm_paged_attn(bt.q, *bt.args(), 1, 40)
    torch.cuda.synchronize()
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


# offsets past 32 bits: pages 2^26 elements apart, 5 GB of cache
@pytest.mark.parametrize("n", [1, 40])
def test_offsets_past_32_bits(q, n):
    bt = Batch([n], [n + 600], 2, 1, 128, "bf16", page=16, seed=8)
    pages, stride = bt.k_cache.shape[0], 1 << 26
    buf = torch.empty(pages * stride + (1 << 20), dtype=bt.dt, device="cuda")
    size, st = (pages, 16, 1, 128), (stride, 128, 128, 1)
    k = torch.as_strided(buf, size, st)
    v = torch.as_strided(buf, size, st, 1 << 19)
    k.copy_(bt.k_cache)
    v.copy_(bt.v_cache)
    bt.k_cache, bt.v_cache = k, v
    assert pages * stride > 2 ** 31
    check(q, bt)


def test_query_views_and_given_buffers(q, route):
    bt = Batch([5, 40], [100, 300], 8, 2, 64, "f16", seed=6)
    wide = torch.zeros(bt.T, 8 + 4, 64, dtype=bt.dt, device="cuda")
    wide[:, :8] = bt.q
    a = check(q, bt)
    b = check(q, bt, query=wide[:, :8])
    assert torch.equal(a, b)
    ws = torch.empty(q.qmm_paged_attn_workspace(8, 2, 64, 40), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(bt.q)
    assert q.qmm_paged_attn(bt.q, *bt.args(), 40, 300, out=out, workspace=ws) is out
    assert torch.equal(a, out)


# a size of one may come with any stride
# every token has the same queries: a stride of zero
@pytest.mark.parametrize("n", [1, 60])
def test_broadcast_queries(q, n):
    bt = Batch([n, n], [n + 30, n + 400], 8, 2, 64, "bf16", seed=3)
    bt.q = bt.q[:1].expand(bt.T, -1, -1)
    check(q, bt)


@pytest.mark.parametrize("n", [1, 40])
def test_strides_of_single_things(q, n):
    bt = Batch([n], [n + 100], 4, 1, 64, seed=4)
    want = check(q, bt)
    k, v = (torch.as_strided(t, t.shape, (t.stride(0), t.stride(1), 5, 1), t.storage_offset()) for t in (bt.k_cache, bt.v_cache))
    bt.k_cache, bt.v_cache = k, v
    assert torch.equal(check(q, bt), want)


# a cache without a page holds no keys: nothing is read
@pytest.mark.parametrize("n", [1, 40])
def test_empty_pool(q, n):
    bt = Batch([n], [0], 4, 2, 64, seed=4)
    none = torch.empty(0, 16, 2, 64, dtype=bt.dt, device="cuda")
    for max_q in (n, 4096):
        out = q.qmm_paged_attn(bt.q, none, none, bt.table, bt.cu_q, bt.kv_len, max_q, 0)
        torch.cuda.synchronize()
        assert (out == 0).all() and q.qmm_device_status() == 0


# the same batch, whatever the caller knows of its lengths; run to run equal
@pytest.mark.parametrize("n", [1, 60])
def test_hints_and_repeats(q, n):
    bt = Batch([n, n], [n + 20, n + 3000], 4, 2, 128, "bf16", seed=n, extra_blocks=9)
    for kw in (dict(), dict(max_kv=0), dict(max_kv=1), dict(max_q=n + 100)):
        out = check(q, bt, **kw)
        again = check(q, bt, **kw)
        assert torch.equal(out, again)


def test_other_stream_and_graph(q):
    bt = Batch([1, 1, 1], [900, 70, 2000], 8, 2, 128, "bf16", seed=12)
    want = check(q, bt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = q.qmm_paged_attn(bt.q, *bt.args(), 1, 2000)
        ws = torch.empty(q.qmm_paged_attn_workspace(8, 2, 128, 1), dtype=torch.uint8, device="cuda")
        buf = torch.empty_like(out)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qmm_paged_attn(bt.q, *bt.args(), 1, 2000, out=buf, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(buf, want)
    # a replay sees the lengths of its own time
    bt.kl = [300, 70, 5]
    for b in (0, 2):
        bt.k64[b], bt.v64[b] = bt.k64[b][:bt.kl[b]], bt.v64[b][:bt.kl[b]]
    bt.kv_len.copy_(torch.tensor(bt.kl, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    ref, tol, _, _ = attention(bt)
    assert ((buf.double() - ref).abs() <= tol).all()
    assert q.qmm_device_status() == 0


# what the host cannot see is checked on the device: nothing out of range is
# touched, the call reports it
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("what", ["page", "page_high", "length", "max_q"])
def test_bad_indices_are_reported(q, n, what):
    bt = Batch([n, n], [n + 300, n + 20], 4, 2, 64, seed=1)
    max_q = n
    if what == "page":
        bt.table[0, 2] = -1
    elif what == "page_high":
        bt.table[0, 2] = bt.k_cache.shape[0]
    elif what == "length":
        bt.kv_len[0] = bt.table.shape[1] * bt.page + 1
    else:
        # 16 rows of the decode kernel hold 8 tokens here, 256 rows of the other 128
        big = 9 if n == 1 else 129
        bt = Batch([big, 1], [big + 5, 30], 4, 2, 64, seed=1)
        max_q = 8 if n == 1 else 128
    q.qmm_paged_attn(bt.q, *bt.args(), max_q, max(bt.kl))
    assert q.qmm_device_status() == 10
    assert q.qmm_device_status() == 0


def test_refusals(q, route):
    bt = Batch([2], [10], 4, 2, 64)
    a = bt.args()
    with pytest.raises(q.QmmError, match="SHAPE"):
        q.qmm_paged_attn(bt.q, *a, 2, 10, scale=0.0)
    with pytest.raises(q.QmmError, match="SHAPE"):
        q.qmm_paged_attn(bt.q, *a, 2, 10, scale=math.inf)
    with pytest.raises(q.QmmError, match="SHAPE"):
        q.qmm_paged_attn(bt.q, *a, 2, 10, window=4, causal=False)
    with pytest.raises(q.QmmError, match="SHAPE"):
        q.qmm_paged_attn(bt.q[:, :3].contiguous(), *a, 2, 10)
    with pytest.raises(q.QmmError, match="SHAPE"):
        q.qmm_paged_attn(bt.q, *a, 2, 10, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        q.qmm_paged_attn(bt.q.half(), *a, 2, 10)
    with pytest.raises(ValueError):
        q.qmm_paged_attn(bt.q, a[0], a[1].transpose(0, 1), *a[2:], 2, 10)
    with pytest.raises(ValueError):
        q.qmm_paged_attn(bt.q, a[0], a[1], a[2].long(), *a[3:], 2, 10)
    with pytest.raises(ValueError):
        q.qmm_paged_attn(bt.q, *a[:4], torch.zeros(2, dtype=torch.int32, device="cuda"), 2, 10)
    with pytest.raises(ValueError):
        q.qmm_paged_attn(bt.q.transpose(0, 1), *a, 2, 10)
    with pytest.raises(ValueError):
        q.qmm_paged_attn(bt.q, *a, 2, 10, out=torch.empty(2, 4, 64, device="cuda"))
    b2 = Batch([2], [10], 4, 2, 64)
    b2.k_cache = b2.k_cache[..., :32]
    b2.v_cache = b2.v_cache[..., :32]
    with pytest.raises(q.QmmError, match="UNSUPPORTED"):
        q.qmm_paged_attn(b2.q[..., :32].contiguous(), *b2.args(), 2, 10)
    assert q.qmm_device_status() == 0
