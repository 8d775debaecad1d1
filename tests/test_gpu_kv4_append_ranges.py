"""qmm_kv4_append where rows hold values that are no numbers, very large or very small: what is not
rotated is copied, and norms keep their relative accuracy."""
import math

import pytest
import torch

from kv4_ref import Batch4, rotate
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
