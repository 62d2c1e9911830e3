"""The prompt kernel's staging in the code that is built: rows come straight
from memory into LDS, and a barrier alone does not wait for such loads, so each
wave has to wait for its own before the barrier that lets the others read them.

The listing of every float16 instance is followed along all of its branches.
No GPU needed, but the compiler."""

import os
import re
import subprocess

import pytest

from dequant_matmul_gptq_amd import build

# What a path knows about the loads to LDS that it has issued.
IDLE, ISSUED, PASSED, LATE = range(4)    # none under way; under way; a barrier passed meanwhile; waited for after it


def _step(state, op, args):
    """The state after one instruction; None: rows that the wave may not have
    are taken to be there (the next ones are asked for, so theirs are in use)."""
    if op.startswith("global_load_lds"):
        return None if state in (PASSED, LATE) else ISSUED
    if op == "s_barrier":
        return {IDLE: IDLE, ISSUED: PASSED, PASSED: PASSED, LATE: IDLE}[state]
    if op == "s_waitcnt" and "vmcnt(0)" in args:
        return {IDLE: IDLE, ISSUED: IDLE, PASSED: LATE, LATE: LATE}[state]
    return state


def _unwaited(lines):
    """Numbers of the loads to LDS that a path reaches with rows of an earlier
    step not waited for before their barrier; and how many such loads there are."""
    code, labels = [], {}
    for line in lines:
        line = line.split(";")[0].strip()
        m = re.match(r"([.\w$]+):$", line)
        if m:
            labels[m.group(1)] = len(code)
        elif line and not line.startswith("."):
            op, _, args = line.partition(" ")
            code.append((op, args.strip()))
    seen, todo, bad = set(), [(0, IDLE)], set()
    while todo:
        at, state = todo.pop()
        if at >= len(code) or (at, state) in seen:
            continue
        seen.add((at, state))
        op, args = code[at]
        if op == "s_endpgm":
            continue
        new = _step(state, op, args)
        if new is None:
            bad.add(at)
            new = ISSUED
        if op.startswith("s_cbranch") or op == "s_branch":
            todo.append((labels[args], new))
        if op != "s_branch":
            todo.append((at + 1, new))
    return sorted(bad), sum(op.startswith("global_load_lds") for op, _ in code)


def test_the_check_itself():
    load, wait, barrier, loop = "global_load_lds_dwordx4 v[0:1], off", "s_waitcnt vmcnt(0)", "s_barrier", "s_cbranch_scc1 .L"
    run = lambda *body: _unwaited([load, ".L:", *body, loop, "s_endpgm"])    # noqa: E731
    assert run(wait, barrier, load) == ([], 2)
    assert run(barrier, load)[0] == [2]                     # no wait
    assert run(barrier, wait, load)[0] == [3]               # too late: the others' rows
    assert run("s_waitcnt vmcnt(1)", barrier, load)[0]      # one still under way
    assert run(wait, barrier, load, barrier)[0] == []       # a barrier inside the step
    assert run("s_cbranch_vccz .M", wait, ".M:", barrier, load)[0]      # on one path only


@pytest.fixture(scope="module", params=(64, 128, 256))
def listing(request, tmp_path_factory):
    try:
        exe = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    out = str(tmp_path_factory.mktemp("listing") / "chunk.s")
    src = os.path.join(build.CSRC, f"attention_chunk_{request.param}.hip")
    subprocess.run([exe, *build.HIPCC_FLAGS, "-S", "--cuda-device-only", src, "-o", out], check=True,
                   capture_output=True)
    with open(out) as f:
        text = f.read()
    m = re.search(rf"^(\w*attention_chunk_kernelILi{request.param}ELi16E\w*):(.*?)^\.Lfunc_end", text, re.M | re.S)
    return m.group(2).split("\n")


def test_staged_rows_are_waited_for(listing):
    bad, loads = _unwaited(listing)
    assert loads >= 4 and not bad
