"""The attention tests of short batches once more on the kernel for many rows, which such
batches do not choose by themselves: rows of padding behind the batch's tokens raise the
bound on a sequence's tokens."""
import math

import pytest
import torch

import test_gpu_paged_attn as short

pytestmark = pytest.mark.gpu


@pytest.fixture
def many():
    import bit_weight_quantized_gb300 as q
    q.load()

    class Padded:
        """The binding with 8192 rows of NaN behind every batch's queries, cut off again."""

        def __getattr__(self, name):
            return getattr(q, name)

        @staticmethod
        def qmm_paged_attn(query, *args, **kw):
            args = list(args)
            args[5] = max(args[5], 8192)
            rows = torch.full((8192, *query.shape[1:]), math.nan, dtype=query.dtype, device=query.device)
            r = q.qmm_paged_attn(torch.cat([query, rows]), *args, **kw)
            return tuple(t[:len(query)] for t in r) if isinstance(r, tuple) else r[:len(query)]

    return Padded()


@pytest.mark.parametrize("n", [1, 130])
@pytest.mark.parametrize("step", [0.02, 0.5])
def test_growing_maximum(many, n, step):
    short.test_growing_maximum(many, n, step)


@pytest.mark.parametrize("scale", [2.0, 1e-3])
@pytest.mark.parametrize("n", [1, 60])
def test_scales(many, scale, n):
    short.test_scales(many, scale, n)


@pytest.mark.parametrize("n", [1, 20, 140])
def test_not_causal(many, n):
    short.test_not_causal(many, n)


@pytest.mark.parametrize("n", [1, 48])
def test_ragged(many, n):
    short.test_ragged(many, n)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_chunks_every_length(many, D, dtype):
    short.test_chunks_every_length(many, D, dtype)


@pytest.mark.parametrize("n,kv", [(1, 40001), (33, 30011)])
def test_long_axis_is_split(many, n, kv):
    short.test_long_axis_is_split(many, n, kv, "f16")


@pytest.mark.parametrize("n", [1, 30])
def test_pages_before_the_window_are_not_read(many, n):
    short.test_pages_before_the_window_are_not_read(many, n)


def test_infinite_and_nan_scores_propagate(many):
    short.test_infinite_and_nan_scores_propagate(many)


@pytest.mark.parametrize("n", [1, 40])
def test_offsets_past_32_bits(many, n):
    short.test_offsets_past_32_bits(many, n)


@pytest.mark.parametrize("n", [1, 40])
def test_strides_of_single_things(many, n):
    short.test_strides_of_single_things(many, n)


@pytest.mark.parametrize("n", [1, 60])
def test_hints_and_repeats(many, n):
    short.test_hints_and_repeats(many, n)
