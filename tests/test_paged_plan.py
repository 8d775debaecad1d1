"""Host-side checks of what qmm_paged_attn launches (no GPU needed).

tests/paged_plan_check.cu compiles the kernel choice and split
(bit_weight_quantized_gb300/csrc/attn.cu) into a host program that prints each launch
in place of making it."""
import os
import shutil
import subprocess
from collections import namedtuple

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
INT_MAX = 2 ** 31 - 1
SMS = 152

Launch = namedtuple("Launch", "few grid warps cluster whole unsplit tile_rows row_tiles min_chunk window part_end scratch")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("paged_plan") / "paged_plan_check")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                    "--expt-relaxed-constexpr", "-o", exe, os.path.join(HERE, "paged_plan_check.cu")],
                   check=True, capture_output=True)
    return exe


@pytest.fixture(scope="module")
def plan(program):
    def run(batches):
        """Launches of (batch, tokens, q_heads, kv_heads, D, page, blocks, window, max_q, max_kv, q_map)."""
        text = "".join(" ".join(str(int(v)) for v in b) + "\n" for b in batches)
        out = subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(out) == 2 * len(batches)
        return [Launch(*map(int, out[2 * i].split()), int(out[2 * i + 1])) for i in range(len(batches))]

    return run


def _decode(batch, heads, keys, D=128, window=0):
    return (batch, batch, 4 * heads, heads, D, 16, -(-keys // 16), window, 1, keys, 1)


# A window that no position of the table reaches past is no window.
def test_window_that_covers_the_table(plan):
    cases = [_decode(4, 2, 304, window=w) for w in (1, 303, 304, 305, INT_MAX)]
    assert [p.window for p in plan(cases)] == [1, 303, 0, 0, 0]


# The first key that a window shows, also of padding (positions below zero) and at the
# ends of the integers.
def test_window_start(program):
    pairs = [(p, w) for p in (-INT_MAX, -5, -3, -2, -1, 0, 1, 62, 63, 64, 65, INT_MAX - 1, INT_MAX)
             for w in (1, 2, 63, 64, 65, INT_MAX - 4, INT_MAX)]
    out = subprocess.run([program, "start"], input="".join(f"{p} {w}\n" for p, w in pairs), capture_output=True,
                         text=True, check=True).stdout.split()
    assert [int(v) for v in out] == [max(0, p - w + 1) for p, w in pairs]


# max_q may be any bound: row tiles cover the batch's tokens and no more, rows are counted in
# 32 bits, and the scratch that the caller was asked for holds the parts.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_map", [0, 1])
def test_row_tiles_of_any_max_q(plan, D, q_map):
    cases = [(b, t, hq, hk, D, 16, 600, 0, max_q, max_kv, q_map) for b in (1, 3, 40) for t in (1, 5, 64, 300, 9000)
             for hq, hk in ((1, 1), (8, 1), (32, 8), (17, 1), (100, 1), (512, 1)) for max_kv in (0, 9000)
             for max_q in (0, 1, 4, 40, t, 8192, 1 << 24, INT_MAX)]
    for c, p in zip(cases, plan(cases)):
        rows = max(1, min(c[8], c[1])) * (c[2] // c[3])
        assert (p.row_tiles - 1) * p.tile_rows < rows <= p.row_tiles * p.tile_rows, (c, p)
        assert p.row_tiles * p.tile_rows < INT_MAX
        assert p.part_end <= p.scratch, (c, p)
        assert p.grid <= (2 if p.few else 1) * SMS or p.whole


# An axis that is split runs on blocks of four warps, which its grid of two blocks per SM
# is made for, whatever the number of items.
@pytest.mark.parametrize("D", [64, 128])
def test_split_decode_runs_on_four_warps(plan, D):
    cases = [_decode(b, h, n, D, w) for h in (1, 2, 8, 16, 32) for n in (300, 520, 600, 1100, 2100, 4096, 30000)
             for b in (1, 7, 29, 33, 58, 66, 100, 115, 128, 133, 200, 256, 400) for w in (0, 700)]
    split = 0
    for c, p in zip(cases, plan(cases)):
        assert p.few
        if not p.whole:
            split += 1
            assert p.warps == 4 and p.cluster == 1, c
            assert p.grid <= 2 * SMS
    assert split > 100


def test_many_short_items_keep_their_narrow_blocks(plan):
    got = plan([_decode(54, 32, 4), _decode(256, 8, 256), _decode(64, 8, 256)])
    assert [p.whole for p in got] == [1, 1, 1]
    assert [p.warps for p in got] == [1, 1, 4]
    assert [p.grid for p in got] == [54 * 32, 2048, 512]
