"""The attention kernels' arithmetic on rows, steps and pages, compiled for the
host, against the same in whole numbers without a limit (no GPU)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    exe = str(tmp_path_factory.mktemp("probe") / "attention_probe")
    cmd = [hipcc, "-std=c++20", "-O1", "-x", "hip", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "dequant_matmul_gptq_amd", "csrc"),
           os.path.join(ROOT, "tests", "host", "attention_probe.cpp"), "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True)

    def ask(what, cases):
        text = "\n".join(" ".join(map(str, (what, *c))) for c in cases)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(cases)
        return got

    return ask


def _first(p, window):
    return max(0, p - window + 1) if window else 0


def test_rows_see_what_the_window_says(probe):
    """Windows up to the largest number, rows before the first token among them."""
    cases = [(n, L, group, window, row0, 16)
             for n, L in ((1, 1), (5, 3), (100, 40), (300, 0), (40, 5000), (64, 2000000000))
             for group in (1, 4) for window in (0, 1, 33, 4096, INT_MAX - 1, INT_MAX)
             for row0 in range(0, n * group, 16)]
    for (n, L, group, window, row0, rows), got in zip(cases, probe("rows", cases)):
        last = min(row0 + rows, n * group) - 1
        lo, hi = L - n + row0 // group, L - n + last // group
        first = _first(L - n, window) // 32
        steps = max((L - 1) // 32 - first, 0) + 1
        assert got == (lo, hi, _first(lo, window), _first(hi, window), first, steps), (n, L, group, window, row0)


def test_lengths_leave_room_to_look_ahead(probe):
    """Lengths bounded by the table, and the tokens looked up two steps past the last one below 2^31."""
    cases = [(L, width, page) for page in (16, 256) for width in (1, 3, 4000, 2 ** 23 - 1, 2 ** 23, 2 ** 27, 2 ** 29)
             for L in (INT_MAX, INT_MAX - 200, INT_MAX - 1500, 5000, 700, 1, 0, -1, -INT_MAX)]
    for (L, width, page), (got,) in zip(cases, probe("length", cases)):
        assert got == max(0, min(L, width * page, INT_MAX - 1023))
        for step in (32, 64):       # of the two kernels: the few-row one looks four turns of a wave ahead
            ahead = 4 if step == 32 else 2
            assert (got // step + 1 + ahead) * step <= INT_MAX


def test_rows_stay_inside_q(probe):
    """Any two numbers in q_start, also ones that are not those of rows."""
    values = (-2 ** 31, -5, 0, 1, 7, 40, 41, 5000, INT_MAX)
    cases = [(q0, q1, tokens) for q0 in values for q1 in values for tokens in (1, 40, 1 << 29)]
    for (q0, q1, tokens), (first, n) in zip(cases, probe("start", cases)):
        want = range(max(q0, 0), max(min(q1, tokens), max(q0, 0)))
        assert (first, n) == (want.start, len(want)) and (n == 0 or first + n <= tokens)
