"""The example layer over a cache in 4 bits (norms, window, first tokens) against a dense
64-bit computation with the keys and values that the cache stands for: prompts in ragged
chunks, then single tokens."""
import os
import sys

import pytest
import torch

from kv4_ref import normed, rotate

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 4)])
def test_prompts_and_steps_equal_the_dense_layer(window, sinks):
    from attention_layer import AttentionLayer, PagedCache4

    import bit_weight_quantized_gb300 as q
    dev = torch.device("cuda")
    layer = AttentionLayer(device=dev, seed=3, norm=True, window=window, sinks=sinks)
    hq, hk, D, page = 8, 2, 128, 16
    chunks = [[130, 3, 47], [129, 1, 0], [16, 40, 5], [1, 1, 1], [1, 1, 1]]
    lens = [sum(c[b] for c in chunks) for b in range(3)]
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    xs = [torch.randn(n, 1024, generator=g, device=dev).half() for n in lens]
    cache = PagedCache4(64, page, hk, D, 3, torch.float16, dev)
    at, got = [0, 0, 0], [[], [], []]
    for new in chunks:
        x = torch.cat([xs[b][at[b]:at[b] + n] for b, n in enumerate(new)])
        y = layer(x, cache, new)
        for b, part in enumerate(torch.split(y, new)):
            got[b].append(part)
            at[b] += new[b]
    # everything that the cache holds
    table, _, kv_len = cache.grow([0, 0, 0])
    cu = torch.tensor([0, lens[0], lens[0] + lens[1], sum(lens)], dtype=torch.int32, device=dev)
    kr, vr = q.qmm_kv4_read(cache.k, cache.v, cache.scales, table, cu, kv_len, sum(lens))
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    # roundings as in the 16-bit layer's test, but for the keys' and values', which are given
    for b in range(3):
        n, x = lens[b], xs[b].double()
        qkv = (x @ layer.qkv.weight.double().T).view(n, hq + 2 * hk, D)
        pos = torch.arange(n, device=dev)
        qr = rotate(normed(qkv[:, :hq], layer.q_norm, 1e-6), pos, layer.cos_sin, False)
        k, v = (t[int(cu[b]):int(cu[b + 1])].double().repeat_interleave(hq // hk, 1) for t in (kr, vr))
        a = torch.einsum("ihd,jhd->hij", qr, k) * D ** -0.5
        hidden = pos[None, :] > pos[:, None]
        if window:
            hidden = hidden | ((pos[None, :] <= pos[:, None] - window) & (pos[None, :] >= sinks))
        a = a.masked_fill(hidden, float("-inf"))
        heads = torch.einsum("hij,jhd->ihd", torch.softmax(a, -1), v)
        add = heads.reshape(n, hq * D) @ layer.out.weight.double().T
        out = torch.cat(got[b]).double()
        assert float((out - x - add).norm() / add.norm()) <= 18 * 2.0 ** -11
        # and the cache holds the layer's keys and values: within half a step, 1 / 15 of the group's
        # largest value at most (and 2% more), and the product's rounding
        for t, ref in ((k, rotate(normed(qkv[:, hq:hq + hk], layer.k_norm, 1e-6), pos, layer.cos_sin, False)), (v, qkv[:, hq + hk:])):
            ref = ref.repeat_interleave(hq // hk, 1).unflatten(-1, (-1, 64))
            near = ref.abs().amax(-1, keepdim=True)
            assert ((t.unflatten(-1, (-1, 64)) - ref).abs() <= near * (1.02 / 15 + 18 * 2.0 ** -11)).all()
