"""The example layer (quantized products, append, attention over the paged cache)
against a dense 64-bit computation of the same layer: prompts in ragged chunks, then
single tokens."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def dense(layer, x, hq, hk, D):
    """The layer on one whole conversation x [n][hidden], causal, in fp64."""
    n = x.shape[0]
    x = x.double()
    qkv = (x @ layer.qkv.weight.double().T).view(n, hq + 2 * hk, D)
    c, s = layer.cos_sin[:n, :D // 2].double()[:, None], layer.cos_sin[:n, D // 2:].double()[:, None]

    def turn(t):
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    qr, k, v = turn(qkv[:, :hq]), turn(qkv[:, hq:hq + hk]), qkv[:, hq + hk:]
    k, v = k.repeat_interleave(hq // hk, 1), v.repeat_interleave(hq // hk, 1)
    a = torch.einsum("ihd,jhd->hij", qr, k) * D ** -0.5
    a = a.masked_fill(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
    heads = torch.einsum("hij,jhd->ihd", torch.softmax(a, -1), v)
    return x + heads.reshape(n, hq * D) @ layer.out.weight.double().T


def test_prompts_and_steps_equal_the_dense_layer():
    from attention_layer import AttentionLayer, PagedCache

    import bit_weight_quantized_gb300 as q
    dev = torch.device("cuda")
    layer = AttentionLayer(device=dev, seed=3)
    hq, hk, D, page = 8, 2, 128, 16
    chunks = [[130, 3, 47], [129, 1, 0], [16, 40, 5], [1, 1, 1], [1, 1, 1]]
    lens = [sum(c[b] for c in chunks) for b in range(3)]
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    xs = [torch.randn(n, 1024, generator=g, device=dev).half() for n in lens]
    cache = PagedCache(64, page, hk, D, 3, torch.float16, dev)
    at, got = [0, 0, 0], [[], [], []]
    for new in chunks:
        x = torch.cat([xs[b][at[b]:at[b] + n] for b, n in enumerate(new)])
        y = layer(x, cache, new)
        for b, part in enumerate(torch.split(y, new)):
            got[b].append(part)
            at[b] += new[b]
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    # Roundings of u = 2^-11 each: the qkv product, the rotated queries and keys, the
    # weights, the heads, the products' operands and y: at most 6 u on what they round;
    # the scores carry 2 u of their size (at most 6 or so here), which the weights take
    # over: 12 u more.
    for b in range(3):
        ref = dense(layer, xs[b], hq, hk, D)
        out = torch.cat(got[b]).double()
        assert float((out - ref).norm() / ref.norm()) <= 18 * 2.0 ** -11
        # the attention's own contribution, too: without the residual
        add = ref - xs[b].double()
        assert float((out - ref).norm() / add.norm()) <= 18 * 2.0 ** -11
