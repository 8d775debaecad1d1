"""The 4-bit cache calls' host checks: each bad argument is refused with its status
before any device work.  Runs without a GPU."""
import ctypes
import os

import pytest
import torch

import bit_weight_quantized_gb300 as q
from bit_weight_quantized_gb300 import build as qbuild

A = 1 << 20   # a 16-byte aligned stand-in address, never dereferenced

host_only = pytest.mark.skipif(os.path.exists("/dev/nvidia0"), reason="host-only checks; a GPU is present")

KV = dict(k=A, v=A, page_stride=1024, slot_stride=64, head_stride=1024, block_table=A, cu_q=A, kv_len=A, num_pages=8,
          page_size=16, blocks=4, batch=2, tokens=5, kv_heads=2, head_dim=128, dtype=1, scales=A, scale_page_stride=64,
          scale_slot_stride=4, scale_head_stride=64)
APPEND = dict(k=A, k_stride=1024, v=A, v_stride=1024, q=A, q_stride=1024, q_out=A, q_heads=8, cos_sin=A, rot=64,
              rope_len=100, interleaved=0, q_norm=A, k_norm=A, eps=1e-6, stream=None)
READ = dict(k_out=A, v_out=A, stream=None)
ATTN = dict(q=A, q_stride=1024, q_heads=8, scale=0.1, causal=1, window=0, sinks=0, out=A, lse=None, max_q=3, max_kv=64,
            workspace=A, workspace_bytes=1 << 30, stream=None)
CALLS = dict(qmm_kv4_append=APPEND, qmm_kv4_read=READ, qmm_kv4_attn=ATTN)

SHAPE, NULL, ALIGN, UNSUPPORTED, DEVICE = 3, 1, 4, 5, 9

KV_CASES = [
    (dict(batch=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(num_pages=-1), SHAPE), (dict(page_size=0), SHAPE),
    (dict(blocks=-1), SHAPE), (dict(kv_heads=0), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(kv_heads=65537), UNSUPPORTED),
    (dict(page_stride=-16), SHAPE), (dict(slot_stride=-16), SHAPE), (dict(head_stride=-16), SHAPE),
    (dict(scale_page_stride=-4), SHAPE), (dict(scale_slot_stride=-4), SHAPE), (dict(scale_head_stride=-4), SHAPE),
    # a stride of one thing is not looked at (valid calls stop at the missing device)
    (dict(num_pages=1, page_stride=3, scale_page_stride=3), DEVICE),
    (dict(page_size=1, slot_stride=3, scale_slot_stride=-3), DEVICE),
    (dict(kv_heads=1, head_stride=-3, scale_head_stride=1), DEVICE),
    (dict(page_stride=1032), ALIGN), (dict(slot_stride=8), ALIGN), (dict(head_stride=24), ALIGN),
    (dict(scale_page_stride=2), ALIGN), (dict(scale_slot_stride=6), ALIGN), (dict(scale_head_stride=1), ALIGN),
    (dict(page_stride=1 << 31), UNSUPPORTED), (dict(scale_page_stride=1 << 40), UNSUPPORTED),
    (dict(page_stride=(1 << 31) - 16), DEVICE), (dict(slot_stride=1 << 27, page_size=17), UNSUPPORTED),
    (dict(slot_stride=1 << 27, page_size=16), DEVICE), (dict(scale_slot_stride=1 << 28), UNSUPPORTED),
    (dict(head_stride=1 << 31), UNSUPPORTED), (dict(scale_head_stride=1 << 31), UNSUPPORTED),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(scales=None), NULL), (dict(block_table=None), NULL),
    (dict(cu_q=None), NULL), (dict(kv_len=None), NULL), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN),
    (dict(scales=A + 4), ALIGN), (dict(scales=A + 8), DEVICE), (dict(head_dim=64, scales=A + 4), DEVICE),
    (dict(head_dim=64, scale_slot_stride=2), DEVICE), (dict(head_dim=64, scale_slot_stride=1), ALIGN),
    (dict(block_table=A + 2), ALIGN), (dict(cu_q=A + 1), ALIGN), (dict(kv_len=A + 2), ALIGN), (dict(batch=0), 0),
    (dict(tokens=0), 0), (dict(), DEVICE),
]
APPEND_CASES = [
    (dict(rot=8), SHAPE), (dict(rot=-16), SHAPE), (dict(rot=144), SHAPE), (dict(rope_len=-1), SHAPE),
    (dict(q_heads=-1), SHAPE), (dict(q_heads=65537), UNSUPPORTED), (dict(eps=-1e-6), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(eps=float("inf")), SHAPE), (dict(k_stride=-8), SHAPE), (dict(q_stride=-8), SHAPE), (dict(k_stride=1), ALIGN),
    (dict(v_stride=4), ALIGN), (dict(q_stride=12), ALIGN), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(cos_sin=None), NULL), (dict(q=None), NULL), (dict(q_out=None), NULL), (dict(k=A + 8), ALIGN),
    (dict(v=A + 8), ALIGN), (dict(q=A + 8), ALIGN), (dict(q_out=A + 8), ALIGN), (dict(cos_sin=A + 4), ALIGN),
    (dict(q_norm=A + 8), ALIGN), (dict(k_norm=A + 2), ALIGN), (dict(cos_sin=None, rot=0), DEVICE),
    (dict(q=None, q_out=None), DEVICE), (dict(q_norm=None, k_norm=None), DEVICE),
]
READ_CASES = [(dict(k_out=None), NULL), (dict(v_out=None), NULL), (dict(k_out=A + 8), ALIGN), (dict(v_out=A + 4), ALIGN)]
ATTN_CASES = [
    (dict(q_heads=7), SHAPE), (dict(q_heads=0), SHAPE), (dict(q_heads=65538), UNSUPPORTED), (dict(window=-1), SHAPE),
    (dict(window=4, causal=0), SHAPE), (dict(sinks=-1, window=4), SHAPE), (dict(sinks=1), SHAPE),
    (dict(sinks=1, window=4), DEVICE), (dict(max_q=-1), SHAPE), (dict(max_kv=-1), SHAPE), (dict(scale=0.0), SHAPE),
    (dict(scale=-1.0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(scale=3e38), SHAPE),
    (dict(q_stride=-8), SHAPE), (dict(q_stride=20), ALIGN), (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(workspace=None), NULL), (dict(q=A + 4), ALIGN), (dict(out=A + 8), ALIGN), (dict(workspace=A + 8), ALIGN),
    (dict(lse=A + 2), ALIGN), (dict(max_q=0), 0),
]
# places of codes are counted in units of the strides' largest power of two
UNIT_CASES = [(dict(num_pages=2 ** 31 - 1, page_stride=48), UNSUPPORTED), (dict(num_pages=2 ** 31 - 1, page_stride=32, slot_stride=32), DEVICE),
              (dict(num_pages=2 ** 20, page_stride=2 ** 20 + 16), UNSUPPORTED), (dict(num_pages=2 ** 18, page_stride=2 ** 20), DEVICE)]


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return q.load()


def call(lib, name, kv, args):
    return getattr(lib, name)(ctypes.byref(q.PagedKV4(*dict(KV, **kv).values())), *args.values())


@host_only
@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("case", range(len(KV_CASES)))
def test_cache_and_batch(lib, name, case):
    kw, want = KV_CASES[case]
    assert call(lib, name, kw, CALLS[name]) == want


@host_only
@pytest.mark.parametrize("name,cases", [("qmm_kv4_append", APPEND_CASES), ("qmm_kv4_read", READ_CASES), ("qmm_kv4_attn", ATTN_CASES)])
def test_arguments(lib, name, cases):
    for kw, want in cases:
        assert call(lib, name, {}, dict(CALLS[name], **kw)) == want, kw


@host_only
@pytest.mark.parametrize("case", range(len(UNIT_CASES)))
def test_units(lib, case):
    kw, want = UNIT_CASES[case]
    assert call(lib, "qmm_kv4_attn", dict(kw, kv_heads=1), ATTN) == want
    assert call(lib, "qmm_kv4_read", dict(kw, kv_heads=1), READ) == DEVICE


@host_only
def test_null_cache(lib):
    for name, args in CALLS.items():
        assert getattr(lib, name)(None, *args.values()) == NULL


@host_only
def test_workspace_sizes_refused(lib):
    for a in ((0, 1, 128, 1), (8, 3, 128, 1), (8, 2, 96, 1), (8, 2, 128, -1), (65538, 2, 128, 1)):
        assert lib.qmm_kv4_attn_workspace(*a) == 0


def test_more_workspace(lib):
    assert lib.qmm_kv4_attn_more_workspace(0, 2048, 32, 8, 128, 2048, 2048, 0) == 0
    assert lib.qmm_kv4_attn_more_workspace(1, 2048, 32, 7, 128, 2048, 2048, 0) == 0
    with pytest.raises(ValueError, match="32 bits"):
        q.qmm_kv4_attn_more_workspace(1, 2048, 32, 8, 128, 2048, 2 ** 31)


def cpu_batch():
    i = torch.zeros(1, dtype=torch.int32)
    return (torch.zeros(2, 16, 2, 32, dtype=torch.uint8), torch.zeros(2, 16, 2, 32, dtype=torch.uint8),
            torch.zeros(2, 16, 2, 2, dtype=torch.float16), i.view(1, 1), torch.zeros(2, dtype=torch.int32), i)


def test_cpu_tensors_are_refused():
    k = torch.zeros(1, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        q.qmm_kv4_append(k, k, *cpu_batch())
    with pytest.raises(ValueError, match="CUDA"):
        q.qmm_kv4_read(*cpu_batch(), 1)
    with pytest.raises(ValueError, match="CUDA"):
        q.qmm_kv4_attn(k, *cpu_batch(), 1)
    with pytest.raises(ValueError, match="negative"):
        q.qmm_kv4_read(*cpu_batch(), -1)
