"""GPU parity of qmm_kv_append against the plain 64-bit form: every stored and
rotated value within one rounding of the exact one, everything else untouched."""
import pytest
import torch

from paged_ref import Batch, U, cos_sin_table, rotate

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
    elif q._fast_append is None:
        pytest.skip("extension not built")


def check(q, bt, rot, interleaved, with_q=True, in_place=False, seed=0):
    """Appends random tokens to bt and compares the whole cache."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 77)
    T, hq, hk, D = bt.T, bt.hq, bt.hk, bt.D
    fused = torch.randn((T, hq + 2 * hk, D), generator=g, device="cuda").to(bt.dt)
    qq, k, v = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:]
    if in_place:
        qq = qq.contiguous()
    cs = cos_sin_table(max(bt.kl) + 1, rot) if rot else None
    want_k, want_v = bt.k_cache.double(), bt.v_cache.double()
    want_k, want_v = want_k.clone(), want_v.clone()
    # positions, and which tokens are padding
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in zip(bt.ql, bt.kl)] + [torch.zeros(0, dtype=torch.long)]).long().cuda()
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(bt.ql)] + [torch.zeros(0, dtype=torch.long)]).long().cuda()
    real = pos >= 0
    # each result is one rounding of a fp32 sum of two products
    size = qq.double().abs().max() * 2 ** -21 if T else 0.0
    kr = rotate(k, pos.clamp(min=0), cs, interleaved)
    qr = rotate(qq, pos.clamp(min=0), cs, interleaved)
    page = bt.table.long()[seq, (pos // bt.page).clamp(min=0)]
    for t in range(T):
        if real[t]:
            want_k[page[t], pos[t] % bt.page] = kr[t]
            want_v[page[t], pos[t] % bt.page] = v[t].double()
    sentinel = torch.full((T, hq, D), 7.0, dtype=bt.dt, device="cuda")
    out = None
    if with_q:
        out = qq if in_place else sentinel.clone()
        before = out.clone()
        assert q.qmm_kv_append(k, v, *bt.args(), q=qq, q_out=out, cos_sin=cs, interleaved=interleaved) is out
    else:
        assert q.qmm_kv_append(k, v, *bt.args(), cos_sin=cs, interleaved=interleaved) is None
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    u = U[bt.dt]

    def near(a, b):
        a, b = a.double(), b.double()
        same = torch.isnan(a) & torch.isnan(b)
        return (same | ((a - b).abs() <= u * b.abs() + size)).all()

    assert near(bt.k_cache, want_k)
    assert torch.equal(torch.nan_to_num(bt.v_cache.double(), nan=9e9), torch.nan_to_num(want_v, nan=9e9))
    if with_q:
        assert near(out[real], qr[real])
        assert torch.equal(out[~real], before[~real])     # padding is left alone
        if rot < D:   # what is not rotated is copied bit for bit
            assert torch.equal(out[real][..., rot:], (qq if not in_place else before)[real][..., rot:])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("part", [0, 16, 32, 64])
def test_rotations(q, D, dtype, interleaved, part):
    rot = min(part, D) if part < 64 else D
    check(q, Batch([1, 7, 40], [30, 7, 300], 8, 2, D, dtype, seed=part), rot, interleaved)


@pytest.mark.parametrize("page,layout", [(1, "hnd"), (7, "nhd"), (16, "hnd"), (24, "gap"), (128, "nhd")])
def test_pages_and_layouts(q, page, layout):
    check(q, Batch([3, 1, 50], [3, 200, 261], 6, 3, 64, "f16", page=page, layout=layout, seed=page), 32, False)


@pytest.mark.parametrize("heads", [(1, 1), (7, 1), (64, 8), (33, 11), (96, 32)])
def test_head_counts(q, heads):
    check(q, Batch([1, 5], [9, 40], *heads, 128, "bf16", seed=heads[0]), 128, False)


@pytest.mark.parametrize("batch", [1, 31, 32, 33, 64, 70])
def test_many_sequences(q, batch):
    check(q, Batch([1] * batch, [1 + (i * 13) % 90 for i in range(batch)], 4, 2, 64, "bf16", seed=batch), 64, True)


def test_empty_sequences_and_padding(q):
    # no new tokens, no keys, tokens before position 0
    check(q, Batch([0, 3, 0, 5, 4, 0], [10, 3, 0, 2, 0, 8], 4, 2, 128, "f16", seed=1), 64, False)
    check(q, Batch([0, 0], [10, 0], 4, 2, 128), 64, False)


def test_tokens_past_the_batch_are_padding(q):
    bt = Batch([2, 3], [20, 30], 4, 2, 64, seed=4)
    g = torch.randn(9, 2, 64, device="cuda").to(bt.dt)
    want = bt.k_cache.clone()
    q.qmm_kv_append(g[:5], g[:5], *bt.args())
    first = bt.k_cache.clone()
    bt.k_cache.copy_(want)
    q.qmm_kv_append(g, g, *bt.args())
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(first.double()), torch.nan_to_num(bt.k_cache.double()))
    assert q.qmm_device_status() == 0


def test_without_queries_and_in_place(q, route):
    check(q, Batch([4, 9], [4, 100], 8, 4, 64, "bf16", seed=2), 64, False, with_q=False)
    check(q, Batch([4, 9], [4, 100], 8, 4, 64, "bf16", seed=2), 64, False, in_place=True)
    check(q, Batch([4, 9], [4, 100], 8, 4, 64, "bf16", seed=2), 32, True, in_place=True)


def test_offsets_past_32_bits(q):
    bt = Batch([20], [620], 2, 1, 128, "bf16", page=16, seed=8)
    pages, stride = bt.k_cache.shape[0], 1 << 26
    buf = torch.empty(pages * stride + (1 << 20), dtype=bt.dt, device="cuda")
    size, st = (pages, 16, 1, 128), (stride, 128, 128, 1)
    k, v = torch.as_strided(buf, size, st), torch.as_strided(buf, size, st, 1 << 19)
    k.copy_(bt.k_cache)
    v.copy_(bt.v_cache)
    bt.k_cache, bt.v_cache = k, v
    assert pages * stride > 2 ** 31
    check(q, bt, 128, False)


@pytest.mark.parametrize("what", ["page", "page_high", "length", "table"])
def test_bad_indices_are_reported(q, what):
    bt = Batch([1, 2], [40, 20], 4, 2, 64, seed=1)
    k = torch.ones(3, 2, 64, device="cuda", dtype=bt.dt)
    before = bt.k_cache.clone()
    cs = cos_sin_table(64, 64)
    if what == "page":
        bt.table[0, 2] = -1
    elif what == "page_high":
        bt.table[0, 2] = bt.k_cache.shape[0]
    elif what == "length":
        bt.kv_len[0] = bt.table.shape[1] * bt.page + 1
    else:
        cs = cs[:39].contiguous()
    q.qmm_kv_append(k, k, *bt.args(), cos_sin=cs)
    assert q.qmm_device_status() == 10
    assert q.qmm_device_status() == 0
    # the good sequence was stored, nothing else changed: 2 slots of 2 heads
    changed = torch.nan_to_num(bt.k_cache.double(), nan=5e5) != torch.nan_to_num(before.double(), nan=5e5)
    assert int(changed.any(-1).sum()) == 4


def test_append_then_attend(q, route):
    """The two calls as a decode loop makes them: token by token equals one chunk."""
    kv, n = 150, 21
    bt = Batch([n], [kv], 8, 2, 128, "bf16", seed=3)
    cs = cos_sin_table(kv, 128)
    fused = torch.randn(n, 12, 128, device="cuda").to(bt.dt)
    qr = q.qmm_kv_append(fused[:, 8:10], fused[:, 10:], *bt.args(), q=fused[:, :8], cos_sin=cs)
    whole = q.qmm_paged_attn(qr, *bt.args(), n, kv)
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    rows = []
    for i in range(n):
        ln = torch.tensor([kv - n + i + 1], dtype=torch.int32, device="cuda")
        args = (bt.k_cache, bt.v_cache, bt.table, one, ln)
        r = q.qmm_kv_append(fused[i:i + 1, 8:10], fused[i:i + 1, 10:], *args, q=fused[i:i + 1, :8], cos_sin=cs)
        rows.append(q.qmm_paged_attn(r, *args, 1, kv))
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    # both sides round every weight (u) and the output (u) once
    one_by_one = torch.cat(rows).double()
    assert ((one_by_one - whole.double()).abs() <= 4 * U[bt.dt] * (1 + whole.double().abs())).all()


def test_refusals(q, route):
    bt = Batch([2], [10], 4, 2, 64)
    k = torch.zeros(2, 2, 64, device="cuda", dtype=bt.dt)
    a = bt.args()
    with pytest.raises(q.QmmError, match="SHAPE"):
        q.qmm_kv_append(k, k, *a, cos_sin=cos_sin_table(20, 24))
    with pytest.raises(q.QmmError, match="SHAPE"):
        q.qmm_kv_append(k, k, *a, cos_sin=cos_sin_table(20, 80))
    with pytest.raises(ValueError):
        q.qmm_kv_append(k, k, *a, cos_sin=cos_sin_table(20, 64).double())
    with pytest.raises(ValueError):
        q.qmm_kv_append(k.half(), k, *a)
    with pytest.raises(ValueError):
        q.qmm_kv_append(k, k[:1], *a)
    with pytest.raises(ValueError):
        q.qmm_kv_append(k, k, *a, q_out=k)
    with pytest.raises(ValueError):
        q.qmm_kv_append(k, k, *a, q=torch.zeros(3, 4, 64, device="cuda", dtype=bt.dt))
    with pytest.raises(ValueError):
        q.qmm_kv_append(k.cpu(), k, *a)
    off = torch.zeros(2 * 2 * 64 + 4, device="cuda", dtype=bt.dt)[4:].view(2, 2, 64)
    with pytest.raises(q.QmmError, match="ALIGN"):
        q.qmm_kv_append(off, k, *a)
    assert q.qmm_device_status() == 0
