"""The workspace of paged attention: a query's answer is enough for its own call
and for all smaller ones (the launch code is compiled for the host; no GPU)."""

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    exe = str(tmp_path_factory.mktemp("probe") / "workspace_probe")
    cmd = [hipcc, "-std=c++20", "-O1", "-x", "hip", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "dequant_matmul_gptq_amd", "csrc"),
           os.path.join(ROOT, "tests", "host", "workspace_probe.cpp"), "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(cases)
        return got

    return run


def _call(cache, q_heads, tokens, batch, max_q, max_kv, window):
    """Sizes as the entry point hands them on (max_q_len within 1 .. tokens)."""
    return (*cache, tokens, q_heads, batch, max(1, min(max_q, tokens)), max_kv, window)


def test_chunks_of_a_prompt(ask):
    """A server's largest chunk and the smaller ones that follow it."""
    for D in (64, 128, 256):
        for kv, heads in ((8, 64), (40, 40), (4, 32), (1, 16)):
            chunks = [8192, 4096, 2048, 1024, 511, 256, 100, 33, 16, 5, 1]
            got = ask([_call((D, 16, kv), heads, n, 1, n, 16384, 0) for n in chunks])
            for need, _ in got:
                assert need <= got[0][1], (D, kv, heads)


@pytest.mark.parametrize("seed", range(4))
def test_an_answer_covers_smaller_calls(ask, seed):
    rng = random.Random(seed)
    log = lambda hi: int(hi ** rng.random() + 0.5)      # noqa: E731
    for _ in range(25):
        kv = rng.choice((1, 2, 3, 5, 8, 10, 32, 40, 100, 300))
        group = rng.choice((1, 2, 4, 5, 8, 16, 17, 33, 64, 71))
        cache = (rng.choice((64, 128, 256)), rng.choice((16, 8, 6, 4)), kv)
        window = rng.choice((0, 0, 1, 100, 1000, 4096))
        top = [log(20000), log(300), log(9000), log(200000)]
        cases = [_call(cache, kv * group, *top, window)]
        for _ in range(400):
            small = [rng.choice((log(x), max(1, x - rng.randrange(40)), x)) for x in top]
            cases.append(_call(cache, kv * group, *small, window))
        got = ask(cases)
        for case, (need, _) in zip(cases, got):
            assert need <= got[0][1], (cases[0], case)
        # no more than the partial results of the most workgroups that run at once
        D = cases[0][0]
        assert got[0][1] <= max(1 << 16, 64 * kv) * (D + 2) * 4


def test_single_tokens_take_no_more_than_they_need(ask):
    cases = [_call((D, bits, 8), 64, batch, batch, 1, 30000, 0) for D in (64, 128, 256) for bits in (16, 4)
             for batch in (1, 7, 64)]
    assert all(need == answer > 0 for need, answer in ask(cases))
