"""The Python binding of the paged cache calls where no device is needed."""
import pytest

import bit_weight_quantized_gb300 as q
from bit_weight_quantized_gb300 import build as qbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    qbuild.build()
    return q.load()


@pytest.mark.parametrize("at", range(4))
@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 1, -2 ** 31 - 1])
def test_sizes_past_32_bits_are_refused(at, big):
    args = [8, 2, 128, 1]
    args[at] = big
    with pytest.raises(ValueError, match="32 bits"):
        q.qmm_paged_attn_workspace(*args)


# something that is neither true nor false: its own error, not one of the interpreter
def test_flags_without_a_truth_value():
    import numpy as np
    import torch
    c = torch.zeros(2, 16, 2, 64, dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    k = torch.zeros(1, 2, 64, dtype=torch.float16)
    both = np.array([True, False])
    with pytest.raises(ValueError):
        q.qmm_kv_append(k, k, c, c, i.view(1, 1), torch.zeros(2, dtype=torch.int32), i, interleaved=both)
    for kw in (dict(causal=both), dict(return_lse=both)):
        with pytest.raises(ValueError):
            q.qmm_paged_attn(k, c, c, i.view(1, 1), torch.zeros(2, dtype=torch.int32), i, 1, **kw)


# compiled against one torch, it is not loaded by another: neither a newer version nor another
# build of the same one
@pytest.mark.parametrize("what", ["version", "build"])
def test_extension_of_another_torch_is_not_loaded(lib, what, monkeypatch):
    import torch
    if qbuild.build_paged() is None:
        pytest.skip("no C++ compiler or headers here")
    try:
        if what == "version":
            monkeypatch.setattr(torch, "__version__", "99.0.0")
        else:
            monkeypatch.setattr(torch.version, "git_version", "0123456789abcdef")
        monkeypatch.setattr(q, "_fast_append", None)
        monkeypatch.setattr(q, "_fast_attn", None)
        q._load_paged(lib)
        assert q._fast_append is None and q._fast_attn is None
        monkeypatch.undo()
        q._load_paged(lib)
        assert q._fast_append is not None and q._fast_attn is not None
    finally:
        monkeypatch.undo()
