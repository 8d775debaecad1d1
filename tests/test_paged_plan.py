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
