"""qmm_paged_attn and qmm_kv_append where lengths, masks, scores and arguments are at
their limits: against the plain 64-bit form within its derived bounds
(tests/paged_ref.py), and refusals."""
import math

import pytest
import torch

from paged_ref import Batch, attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_weight_quantized_gb300 as q
    q.load()
    return q


def attend(q, bt, window=0, causal=True, max_q=None, max_kv=None, pad=0):
    """out, lse of one call; `pad` rows of NaN follow the batch's queries, which belong to
    no sequence and whose output must stay as it was."""
    query = bt.q
    if pad:
        query = torch.cat([bt.q, torch.full((pad, bt.hq, bt.D), math.nan, dtype=bt.dt, device=bt.q.device)])
    out = torch.full_like(query, 7.0)
    got, lse = q.qmm_paged_attn(query, *bt.args(), (max(bt.ql) if max_q is None else max_q),
                                max(bt.kl) if max_kv is None else max_kv, causal=causal, window=window,
                                return_lse=True, out=out)
    assert got is out
    torch.cuda.synchronize()
    assert q.qmm_device_status() == 0
    assert (out[bt.T:] == 7.0).all()
    return out[:bt.T], lse[:bt.T]


def check(q, bt, window=0, causal=True, **kw):
    out, lse = attend(q, bt, window, causal, **kw)
    ref, tol, ls, ltol = attention(bt, None, causal, window)
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs out of bounds, first at {bad.nonzero()[0].tolist()}"
    empty = torch.isinf(ls)
    assert torch.equal(lse == -math.inf, empty) and (out[empty] == 0).all()
    assert ((lse.double() - ls).abs()[~empty] <= ltol[~empty]).all()
    return out


# the largest window there is; the tiles hold tokens before position 0, too
@pytest.mark.parametrize("n", [3, 50])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5])
def test_window_of_any_size_beside_padding(q, n, window):
    bt = Batch([n, n + 3, 2 * n], [n // 2, 3, n + 300], 8, 2, 128, "bf16", seed=n)
    check(q, bt, window=window)
    check(q, bt, window=window, pad=4000, max_q=4000)
