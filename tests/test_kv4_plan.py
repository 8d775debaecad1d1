"""Host-side checks of what qmm_kv4_attn launches (no GPU needed).

tests/kv4_plan_check.cu compiles the kernel choice and split
(bit_weight_quantized_gb300/csrc/kv4_attn.cu) into a host program that prints each launch
in place of making it."""
import os
import random
import shutil
import subprocess
from collections import namedtuple

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
INT_MAX = 2 ** 31 - 1
SMS = 152

Launch = namedtuple("Launch", "few grid warps cluster whole unsplit tile_rows row_tiles min_chunk window sinks part_end scratch")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("kv4_plan") / "kv4_plan_check")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                    "--expt-relaxed-constexpr", "-o", exe, os.path.join(HERE, "kv4_plan_check.cu")],
                   check=True, capture_output=True)

    def run(batches):
        """Launches of (batch, tokens, q_heads, kv_heads, D, page, blocks, window, sinks, max_q, max_kv, q_map), with
        the scratch to convert keys once where a 13th number says so."""
        text = "".join(" ".join(str(int(v)) for v in (*b, 0)[:13]) + "\n" for b in batches)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(out) == 2 * len(batches)
        return [Launch(*map(int, out[2 * i].split()), int(out[2 * i + 1])) for i in range(len(batches))]

    return run


def decode(batch, heads, keys, group=4, D=128, window=0, sinks=0):
    return (batch, batch, group * heads, heads, D, 16, -(-keys // 16), window, sinks, 1, keys, 1)


def test_window_that_covers_the_table(plan):
    got = plan([decode(4, 2, 304, window=w, sinks=s) for w, s in ((1, 5), (303, 1), (304, 1), (305, 2), (INT_MAX, INT_MAX))])
    assert [(p.window, p.sinks) for p in got] == [(1, 5), (303, 1), (0, 0), (0, 0), (0, 0)]


def test_forms(plan):
    one, batch, long_one, many, chunk = plan([
        decode(1, 8, 2000), decode(64, 8, 700), decode(1, 8, 131072), decode(64, 32, 200),
        (1, 512, 32, 8, 128, 16, 1024, 0, 0, 512, 16384, 1)])
    assert one.few and one.whole and one.cluster == 8 and one.warps == 8 and one.grid == 64 and one.tile_rows == 8
    assert batch.few and batch.whole and batch.cluster == 1 and batch.warps == 4 and batch.grid == 512
    assert long_one.few and not long_one.whole and long_one.grid == 4 * SMS
    assert many.whole and many.grid == 2048 and many.warps == 4
    assert not chunk.few and not chunk.whole and chunk.grid == SMS and chunk.tile_rows == 256


# The kernel for many rows needs a tensor map of the queries.
def test_queries_without_a_tensor_map(plan):
    a, b = plan([(8, 4000, 32, 8, 128, 16, 256, 0, 0, 500, 4000, 0), (2, 600, 129, 1, 64, 16, 256, 0, 0, 300, 4000, 1)])
    assert a.few and b.few


# Keys are converted once for long prompts without first tokens, where there is scratch.
def test_converted_keys(plan):
    prompt = (1, 2048, 32, 8, 128, 16, 128, 0, 0, 2048, 2048, 1)
    got = plan([prompt, (*prompt, 1), (*prompt[:7], 1990, 0, *prompt[9:], 1), (*prompt[:7], 100, 0, *prompt[9:], 1),
                (*prompt[:7], 1990, 4, *prompt[9:], 1),
                (*prompt[:9], 100, 2048, 1, 1), (*prompt[:10], 0, 1, 1), (16, 2063, *prompt[2:], 1)])
    assert [p.few for p in got] == [0, 2, 2, 0, 0, 0, 0, 0]
    assert got[1].scratch - got[0].scratch >= 2 * 2 * 2048 * 8 * 128


# Partial results stay inside the scratch that is asked for, and numbers in their ranges,
# whatever the batch.
def test_scratch_and_ranges(plan):
    r = random.Random(5)
    batches = []
    for _ in range(3000):
        hk = r.choice([1, 2, 3, 8, 32, 128])
        group = r.choice([1, 2, 5, 8, 12, 16, 128, 200])
        batch = r.choice([1, 2, 7, 64, 300, 5000])
        max_q = r.choice([0, 1, 2, 5, 17, 300, 5000, INT_MAX])
        tokens = r.randint(batch, batch * 50)
        page = r.choice([1, 7, 16, 128])
        blocks = r.choice([0, 1, 5, 1000, 100000])
        window = r.choice([0, 0, 1, 33, 1000, INT_MAX])
        sinks = r.choice([0, 1, 4, 1000, INT_MAX]) if window else 0
        max_kv = r.choice([0, 1, 100, 10000, INT_MAX])
        if (min(max_q, tokens) * group // 8 + 1) * batch > INT_MAX or tokens * group > INT_MAX:
            continue
        batches.append((batch, tokens, hk * group, hk, r.choice([64, 128]), page, blocks, window, sinks, max_q, max_kv, 1,
                        r.choice([0, 1])))
    plans = plan(batches)
    assert {p.few for p in plans} == {0, 1, 2}
    for b, p in zip(batches, plans):
        assert 0 <= p.part_end <= p.scratch, b
        assert 1 <= p.grid <= INT_MAX and p.cluster in (1, 2, 4, 8), b
        assert p.row_tiles * p.tile_rows >= min(max(b[9], 1), b[1]) * (b[2] // b[3]), b
        if p.few == 1:
            assert p.tile_rows in (8, 16) and p.warps in (4, 8) and (p.cluster == 1 or p.warps == 8), b
        else:
            assert p.tile_rows <= 256 and p.tile_rows % (b[2] // b[3]) == 0, b
