"""The paged cache calls' host checks: each bad argument is refused with its status
before any device work.  Runs without a GPU."""
import ctypes
import os

import pytest

import bit_weight_quantized_gb300 as q
from bit_weight_quantized_gb300 import build as qbuild

A = 1 << 20   # a 16-byte aligned stand-in address, never dereferenced

pytestmark = pytest.mark.skipif(os.path.exists("/dev/nvidia0"), reason="host-only checks; a GPU is present")

KV = dict(k=A, v=A, page_stride=2048, slot_stride=128, head_stride=2048, block_table=A, cu_q=A, kv_len=A,
          num_pages=8, page_size=16, blocks=4, batch=2, tokens=5, kv_heads=2, head_dim=128, dtype=1)
APPEND = dict(k=A, k_stride=1024, v=A, v_stride=1024, q=A, q_stride=1024, q_out=A, q_heads=8, cos_sin=A, rot=128,
              rope_len=100, interleaved=0, stream=None)
ATTN = dict(q=A, q_stride=1024, q_heads=8, scale=0.1, causal=1, window=0, out=A, lse=None, max_q=3, max_kv=64,
            workspace=A, workspace_bytes=1 << 30, stream=None)

SHAPE, NULL, ALIGN, UNSUPPORTED, DEVICE = 3, 1, 4, 5, 9

KV_CASES = [
    (dict(batch=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(num_pages=-1), SHAPE), (dict(page_size=0), SHAPE),
    (dict(blocks=-1), SHAPE), (dict(kv_heads=0), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(head_dim=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(page_stride=-8), SHAPE), (dict(slot_stride=-8), SHAPE), (dict(head_stride=-8), SHAPE),
    # a stride of one thing is not looked at (valid calls stop at the missing device)
    (dict(num_pages=1, page_stride=3), DEVICE), (dict(page_size=1, slot_stride=3), DEVICE),
    (dict(kv_heads=1, head_stride=-3), DEVICE),
    (dict(page_stride=2044), ALIGN), (dict(slot_stride=4), ALIGN), (dict(head_stride=1), ALIGN),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(block_table=None), NULL), (dict(cu_q=None), NULL),
    (dict(kv_len=None), NULL), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(block_table=A + 2), ALIGN),
    (dict(cu_q=A + 1), ALIGN), (dict(kv_len=A + 2), ALIGN), (dict(batch=0), 0), (dict(tokens=0), 0), (dict(), DEVICE),
]
APPEND_CASES = [
    (dict(rot=8), SHAPE), (dict(rot=-16), SHAPE), (dict(rot=144), SHAPE), (dict(rope_len=-1), SHAPE),
    (dict(q_heads=-1), SHAPE), (dict(k_stride=-8), SHAPE), (dict(q_stride=-8), SHAPE), (dict(k_stride=1), ALIGN), (dict(v_stride=4), ALIGN), (dict(q_stride=12), ALIGN),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(cos_sin=None), NULL), (dict(q=None), NULL),
    (dict(q_out=None), NULL), (dict(k=A + 8), ALIGN), (dict(v=A + 8), ALIGN), (dict(q=A + 8), ALIGN),
    (dict(q_out=A + 8), ALIGN), (dict(cos_sin=A + 4), ALIGN), (dict(cos_sin=None, rot=0), DEVICE),
    (dict(q=None, q_out=None), DEVICE),
]
ATTN_CASES = [
    (dict(q_heads=7), SHAPE), (dict(q_heads=0), SHAPE), (dict(window=-1), SHAPE), (dict(window=4, causal=0), SHAPE),
    (dict(max_q=-1), SHAPE), (dict(max_kv=-1), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(scale=3e38), SHAPE), (dict(q_stride=-8), SHAPE), (dict(q_stride=20), ALIGN),
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(workspace=None), NULL), (dict(q=A + 4), ALIGN),
    (dict(out=A + 8), ALIGN), (dict(workspace=A + 8), ALIGN), (dict(lse=A + 2), ALIGN), (dict(max_q=0), 0),
]


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return q.load()


def call(lib, name, kv, args):
    return getattr(lib, name)(ctypes.byref(q.PagedKV(*dict(KV, **kv).values())), *args.values())


@pytest.mark.parametrize("name", ["qmm_kv_append", "qmm_paged_attn"])
@pytest.mark.parametrize("case", range(len(KV_CASES)))
def test_cache_and_batch(lib, name, case):
    kw, want = KV_CASES[case]
    assert call(lib, name, kw, APPEND if name == "qmm_kv_append" else ATTN) == want


@pytest.mark.parametrize("case", range(len(APPEND_CASES)))
def test_append_arguments(lib, case):
    kw, want = APPEND_CASES[case]
    assert call(lib, "qmm_kv_append", {}, dict(APPEND, **kw)) == want


@pytest.mark.parametrize("case", range(len(ATTN_CASES)))
def test_attention_arguments(lib, case):
    kw, want = ATTN_CASES[case]
    assert call(lib, "qmm_paged_attn", {}, dict(ATTN, **kw)) == want


def test_extension_is_built_and_loaded(lib):
    if qbuild.build_paged() is None:
        pytest.skip("no C++ compiler or headers here")
    assert q._fast_append is not None and q._fast_attn is not None
    assert q._append_addr and q._attn_addr and q._scratch_addr


def test_null_cache(lib):
    assert lib.qmm_kv_append(None, *APPEND.values()) == NULL
    assert lib.qmm_paged_attn(None, *ATTN.values()) == NULL


def test_workspace_sizes_refused(lib):
    for a in ((0, 1, 128, 1), (8, 3, 128, 1), (8, 2, 96, 1), (8, 2, 128, -1)):
        assert lib.qmm_paged_attn_workspace(*a) == 0


def test_status_string(lib):
    assert b"index" in lib.qmm_status_string(10)


def test_cpu_tensors_are_refused():
    import torch
    c = torch.zeros(2, 16, 2, 64, dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    k = torch.zeros(1, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        q.qmm_kv_append(k, k, c, c, i.view(1, 1), torch.zeros(2, dtype=torch.int32), i)
    with pytest.raises(ValueError):
        q.qmm_paged_attn(k, c, c, i.view(1, 1), torch.zeros(2, dtype=torch.int32), i, 1)
