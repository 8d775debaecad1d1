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
