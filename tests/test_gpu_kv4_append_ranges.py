"""qmm_kv4_append where rows hold values that are no numbers, very large or very small: what is not
rotated is copied, and norms keep their relative accuracy."""
import math

import pytest
import torch

from kv4_ref import Batch4, pack, patterns, quantize, rotate, values
from paged_ref import cos_sin_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_weight_quantized_gb300 as q
    q.load()
    return q


def status(q):
    torch.cuda.synchronize()
    return q.qmm_device_status()


# Elements rot .. D - 1 without a norm: the same bits, whatever their neighbours hold.
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 32), (64, 48), (128, 16), (128, 64), (128, 96), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_what_is_not_rotated_is_copied(q, dtype, D, rot, interleaved):
    bt = Batch4([5], [9], 6, 2, D, dtype, fill=False)
    g = torch.Generator(device="cuda")
    g.manual_seed(rot)
    qkv = torch.randn((5, 10, D), generator=g, device="cuda").to(bt.dt)
    x, odd = qkv[:, :6], [math.inf, -math.inf, math.nan, -math.nan, -0.0, torch.finfo(bt.dt).max, torch.finfo(bt.dt).tiny / 4]
    for i, at in enumerate(range(rot, D, 5)):
        x[i % 5, i % 6, at] = odd[i % len(odd)]
    x[1, 2, rot:] = -0.0
    cs = cos_sin_table(9, rot) if rot else None
    got = q.qmm_kv4_append(qkv[:, 6:8], qkv[:, 8:], *bt.args(), q=x, cos_sin=cs, interleaved=interleaved)
    assert status(q) == 0
    assert torch.equal(got[..., rot:].contiguous().view(torch.int16), x[..., rot:].contiguous().view(torch.int16))
    # and the rest is rotated, within a rounding
    if rot:
        ref = rotate(x[..., :rot], torch.arange(4, 9, device="cuda"), cs, interleaved)
        near = x[..., :rot].double().abs().amax(-1, keepdim=True)
        assert ((got[..., :rot].double() - ref).abs() <= torch.finfo(bt.dt).eps / 2 * ref.abs() + 2.0 ** -22 * near).all()


# Heads so large or small that their squares are no fp32 numbers, beside ordinary ones in a token.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,size,eps", [
    ("bf16", 2.0 ** 62, 1e-6), ("bf16", 1e20, 1e-6), ("bf16", 1e37, 1e-6), ("bf16", 1e20, 0.0), ("bf16", 1e-18, 0.0),
    ("bf16", 1e-25, 0.0), ("bf16", 1e-37, 0.0), ("bf16", 1e-25, 1e-6), ("bf16", 1e-25, 1e-45), ("bf16", 1e-25, 1e-30),
    ("bf16", 1e15, 1e37), ("f16", 1e4, 1e-6), ("f16", 1e-6, 0.0)])
@pytest.mark.parametrize("rot", [0, 32, 64])
def test_norms_of_large_and_small_heads(q, dtype, size, eps, D, rot):
    bt = Batch4([6], [9], 6, 2, D, dtype, fill=False)
    g = torch.Generator(device="cuda")
    g.manual_seed(D + rot)
    qkv = torch.randn((6, 10, D), generator=g, device="cuda").double()
    qkv[::2, ::2] *= size
    qkv[1, 5] *= size
    qkv[2, 4, ::2] = 0.0
    qkv = qkv.to(bt.dt)
    w = [(1 + torch.randn(D, generator=g, device="cuda") / 4).to(bt.dt) for _ in range(2)]
    cs = cos_sin_table(9, rot) if rot else None
    got = q.qmm_kv4_append(qkv[:, 6:8], qkv[:, 8:], *bt.args(), q=qkv[:, :6], cos_sin=cs, q_norm=w[0], k_norm=w[1], eps=eps)
    k = q.qmm_kv4_read(*bt.args(), 6)[0]
    assert status(q) == 0
    for x, weight, y in ((qkv[:, :6], w[0], got), (qkv[:, 6:8], w[1], k)):
        eps32 = float(torch.tensor(eps))                         # what the call takes
        x = x.double()
        ref = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps32) * weight.double()
        ref = rotate(ref, torch.arange(3, 9, device="cuda"), cs, False)
        # as with ordinary heads: D / 2 + 8 roundings of 2^-24, a rotated value below 2 max |x|; the output's rounding,
        # half a step of the type's smallest numbers at least
        f = torch.finfo(bt.dt)
        tol = f.eps / 2 * ref.abs() + 2 * (D / 2 + 8) * 2.0 ** -24 * ref.abs().amax(-1, keepdim=True) + f.tiny * f.eps / 2
        if y is k:                                               # read back: within half a step, (hi - lo) / 15 and 9 / 8 of it
            near = ref.unflatten(-1, (-1, 64))
            step = (near.amax(-1).clamp(min=0) - near.amin(-1).clamp(max=0)) / 15 * 9 / 8 + 2.0 ** (-129 if dtype == "bf16" else -20)
            tol = tol + step.repeat_interleave(64, -1) * (0.5 + 2.0 ** -6)
        assert ((y.double() - ref).abs() <= tol).all()


# Groups whose (hi - lo) / 15 is a number of the scale's bits, or above one by less than fp32 can tell.
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_next_to_a_step(q, dtype, D):
    bt = Batch4([60], [60], 1, 1, D, dtype, fill=False)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    hi, size = torch.arange(1, 16, device="cuda").double(), (0.25 if dtype == "bf16" else 128.0)
    v = torch.zeros((60, 1, D), dtype=torch.float64, device="cuda")
    for i in range(60):
        top = float(hi[i % 15]) * (15 if i < 30 else 1) * size
        x = torch.rand(D, generator=g, device="cuda").double() * top
        x[::64] = top
        if i % 2:
            x[7::64] = -top * 2.0 ** (i % 15 - 30) if dtype == "bf16" else -2.0 ** -24
        v[i, 0] = -x if i % 4 > 1 else x
    v = v.to(bt.dt)
    q.qmm_kv4_append(v, v, *bt.args())
    got = q.qmm_kv4_read(*bt.args(), 60)[1]
    assert status(q) == 0
    c, s, z = quantize(v)
    seq_page = bt.table.long()[0, torch.arange(60, device="cuda") // bt.page]
    pats = bt.scales.view(torch.int16)[seq_page, torch.arange(60, device="cuda") % bt.page][..., D // 64:]
    assert torch.equal(pats, patterns(s, z, bt.dt).view(torch.int16))
    assert torch.equal(got.double(), values(pack(c), patterns(s, z, bt.dt)))
