"""Parts that a row of logits is cut into, and how many of them the join reads.
The launch code is compiled for the host; no GPU needed."""

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = 1 << 22


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    exe = str(tmp_path_factory.mktemp("probe") / "logprob_parts_probe")
    cmd = [hipcc, "-std=c++20", "-O1", "-x", "hip", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "dequant_matmul_gptq_amd", "csrc"),
           os.path.join(ROOT, "tests", "host", "logprob_parts_probe.cpp"), "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return run


def test_no_row_has_more_parts_than_the_join_reads(parts):
    rng = random.Random(0)
    vocabularies = [*range(MOST - 40, MOST + 1), *(rng.randrange(1, MOST + 1) for _ in range(400)),
                    *(n * 1024 * 4 + d for n in (1, 15, 16, 255, 256, 257, 512, 1023) for d in range(-4, 5))]
    cases = [(rows, v, bits) for v in vocabularies for bits in (16, 32) for rows in (1, 2, 3, 7, 64, 600, MOST - 1)]
    got = parts(cases)
    assert len(got) == len(cases)
    for case, (whole, other, most) in zip(cases, got):
        size = 128 // case[2]                       # elements of 16 bytes
        longest = 256 * 16 * size                   # of a part: 256 threads with 16 groups
        assert -(-case[1] // longest) <= whole <= most, case
        assert -(-(case[1] + size - 1) // longest) <= other <= most, case
    # the longest float32 rows that start inside a group have one more than a join has threads
    assert [parts([(2, v, 32)])[0][:2] for v in (MOST - 3, MOST - 2, MOST)] == [(256, 256), (256, 257), (256, 257)]
