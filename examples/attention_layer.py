"""The attention block of a decoder layer on quantized weights, prompts and decode
steps, with the library's calls only (torch allocates, adds the residual and keeps
the page lists):

    qkv  = x . W_qkv^T                 qmm_gemm (17 tokens or more), qmm_gemv
    append, rotate                     qmm_kv_append
    attend over the paged cache        qmm_paged_attn
    y    = x + heads . W_o^T           qmm_gemm / qmm_gemv

or, over a cache in 4 bits, with queries and keys normed per head, a window and first
tokens that stay visible: qmm_kv4_append and qmm_kv4_attn.

    python examples/attention_layer.py

Three conversations share one pool of pages.  Their prompts go in in chunks, all in
one batch however ragged; then every step decodes one token of each.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_quantized_gb300 as q  # noqa: E402

BITS, GROUP = 4, 128


class QuantizedLinear:
    """y = x . W^T for a float weight [N][K], stored as 4-bit codes with a scale and a
    zero per group of 128."""

    def __init__(self, weight):
        N, K = weight.shape
        w = weight.float().view(N, K // GROUP, GROUP)
        # the grid holds zero: the zero point is a code of its own, 0 to 255
        lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        scale = ((hi - lo) / (2 ** BITS - 1)).clamp(min=1e-6).half()
        zero = (-lo / scale.float()).round().clamp(0, 255)
        codes = (w / scale.float()[..., None] + zero[..., None]).round().clamp(0, 2 ** BITS - 1)
        self.packed = q.qmm_pack(codes.view(N, K).to(torch.uint8).contiguous(), BITS)
        self.scales, self.zeros = scale.contiguous(), zero.to(torch.uint8).contiguous()
        # the weight that the codes stand for (for comparisons only)
        self.weight = ((codes - zero[..., None]) * scale.float()[..., None]).view(N, K)

    def __call__(self, x):
        f = q.qmm_gemm if x.shape[0] >= 17 else q.qmm_gemv
        return f(x, self.packed, BITS, GROUP, self.scales, self.zeros)


class PagedCache:
    """Keys and values of one layer in pages handed out as conversations grow."""

    def __init__(self, pages, page, kv_heads, head_dim, batch, dtype, device):
        # heads outside: a page's keys of one head are consecutive
        self.k, self.v = (torch.zeros(pages, kv_heads, page, head_dim, dtype=dtype, device=device).permute(0, 2, 1, 3)
                          for _ in range(2))
        self.page, self.free, self.lists = page, list(range(pages)), [[] for _ in range(batch)]
        self.lengths = [0] * batch

    def grow(self, new):
        """Room for new[b] more keys of conversation b; the batch's tables."""
        for b, n in enumerate(new):
            self.lengths[b] += n
            while len(self.lists[b]) * self.page < self.lengths[b]:
                self.lists[b].append(self.free.pop())
        width = max(len(p) for p in self.lists)
        table = torch.tensor([p + [0] * (width - len(p)) for p in self.lists], dtype=torch.int32)
        cu = torch.zeros(len(new) + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(new), 0)
        dev = self.k.device
        return table.to(dev), cu.to(dev), torch.tensor(self.lengths, dtype=torch.int32, device=dev)


class PagedCache4(PagedCache):
    """The same in 4 bits: codes, and a scale pattern per 64 values."""

    def __init__(self, pages, page, kv_heads, head_dim, batch, dtype, device):
        super().__init__(0, page, kv_heads, head_dim, batch, dtype, device)
        self.k, self.v = (torch.zeros(pages, kv_heads, page, head_dim // 2, dtype=torch.uint8, device=device).permute(0, 2, 1, 3)
                          for _ in range(2))
        self.scales = torch.zeros(pages, kv_heads, page, head_dim // 32, dtype=dtype, device=device).permute(0, 2, 1, 3)
        self.free = list(range(pages))


class AttentionLayer:
    """norm: queries and keys are normed per head; window, sinks: tokens that a token sees (both
    over a cache in 4 bits)."""

    def __init__(self, hidden=1024, q_heads=8, kv_heads=2, head_dim=128, max_len=4096, device="cuda", seed=0, norm=False,
                 window=0, sinks=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.heads, self.kv_heads, self.D = q_heads, kv_heads, head_dim

        def weight(n, k):
            return torch.randn(n, k, generator=g, device=device) * k ** -0.5

        self.qkv = QuantizedLinear(weight((q_heads + 2 * kv_heads) * head_dim, hidden))
        self.out = QuantizedLinear(weight(hidden, q_heads * head_dim))
        freq = 10000.0 ** (-torch.arange(head_dim // 2, device=device, dtype=torch.float64) * 2 / head_dim)
        ang = torch.arange(max_len, device=device, dtype=torch.float64)[:, None] * freq
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        self.window, self.sinks = window, sinks
        self.q_norm = self.k_norm = None
        if norm:
            self.q_norm, self.k_norm = (1 + torch.randn(2, head_dim, generator=g, device=device) / 4).half()

    def __call__(self, x, cache, new):
        """x [tokens][hidden] (fp16): new[b] tokens of every conversation b, packed."""
        T, hq, hk = x.shape[0], self.heads, self.kv_heads
        table, cu_q, kv_len = cache.grow(new)
        qkv = self.qkv(x).view(T, hq + 2 * hk, self.D)
        if isinstance(cache, PagedCache4):
            cached = cache.k, cache.v, cache.scales, table, cu_q, kv_len
            turned = q.qmm_kv4_append(qkv[:, hq:hq + hk], qkv[:, hq + hk:], *cached, q=qkv[:, :hq], cos_sin=self.cos_sin,
                                      q_norm=self.q_norm, k_norm=self.k_norm)
            heads = q.qmm_kv4_attn(turned, *cached, max(new), max(cache.lengths), window=self.window, sinks=self.sinks)
            return x + self.out(heads.view(T, hq * self.D))
        rotated = q.qmm_kv_append(qkv[:, hq:hq + hk], qkv[:, hq + hk:], cache.k, cache.v, table, cu_q, kv_len,
                                  q=qkv[:, :hq], cos_sin=self.cos_sin)
        heads = q.qmm_paged_attn(rotated, cache.k, cache.v, table, cu_q, kv_len, max(new), max(cache.lengths))
        return x + self.out(heads.view(T, hq * self.D))


def run(layer, kind):
    dev = torch.device("cuda")
    prompts, chunk, steps = [700, 45, 300], 256, 16
    cache = kind(128, 16, 2, 128, len(prompts), torch.float16, dev)
    left = list(prompts)
    while any(left):
        new = [min(n, chunk) for n in left]
        left = [a - b for a, b in zip(left, new)]
        layer(torch.randn(sum(new), 1024, device=dev).half(), cache, new)
    x = torch.randn(len(prompts), 1024, device=dev).half()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(steps):
        x = layer(x, cache, [1] * len(prompts))
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / steps
    assert q.qmm_device_status() == 0
    print(f"{kind.__name__}: prompts of {prompts} tokens in, {steps} steps of {len(prompts)} tokens: {t * 1e6:.0f} us a step "
          f"(one layer, host work and page lists included); keys now {cache.lengths}")


def main():
    run(AttentionLayer(), PagedCache)
    run(AttentionLayer(norm=True, window=512, sinks=4), PagedCache4)


if __name__ == "__main__":
    main()
