"""Registers that the compiler spills in the views' few-row kernels, in the code
that is built. Where a branch left some lanes off and a register is stored to
scratch memory before they are on again, those lanes lack it when it is loaded
back: hipcc 7.2 did that around loads that only some lanes made, and the address
made of it was then anything. (Registers for scalars take lanes by number and
do not ask which are on.)

The listing of every instance is looked over. No GPU needed, but the compiler."""

import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from dequant_matmul_gptq_amd import build

SOURCES = [f"attention_view_few_{d}.hip" for d in (64, 128, 256)]


def _stores_before_restore(lines):
    """Stores to scratch memory between a label and the restoring of the lanes there."""
    bad, since = [], None
    for line in lines:
        op = line.split(";")[0].strip()
        if re.match(r"[.\w$]+:$", op):
            since = []
        elif since is not None and op:
            if re.match(r"s_or_b64 exec, exec, ", op):
                bad += since
                since = None
            elif re.match(r"s_c?branch|s_endpgm|s_barrier|s_\w+ exec|s_\w+saveexec", op):
                since = None
            elif op.startswith(("scratch_store", "v_accvgpr_write")):
                since.append(op)
    return bad


def test_the_check_itself():
    store, restore = "scratch_store_dwordx2 off, v[44:45], off offset:324", "s_or_b64 exec, exec, s[6:7]"
    assert _stores_before_restore([".L:", "s_mov_b32 s1, s2", store, restore]) == [store]
    assert _stores_before_restore([".L:", restore, store]) == []
    assert _stores_before_restore([".L:", "v_mov_b32 v1, v2", store, "s_cbranch_vccz .M", ".M:", restore]) == []
    assert _stores_before_restore([".L: ; %bb", "v_accvgpr_write_b32 a1, v2 ; Folded", restore]) == ["v_accvgpr_write_b32 a1, v2"]


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    try:
        exe = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    to = tmp_path_factory.mktemp("listing")

    def make(name):
        out = str(to / (name + ".s"))
        subprocess.run([exe, *build.HIPCC_FLAGS, "-S", "--cuda-device-only", os.path.join(build.CSRC, name), "-o", out],
                       check=True, capture_output=True)
        with open(out) as f:
            return f.read()

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        return "".join(ex.map(make, SOURCES))


def test_no_register_is_stored_while_lanes_are_off(listings):
    kernels = re.findall(r"^(_Z\w*attention_few_kernel\w*):(.*?)^\.Lfunc_end", listings, re.M | re.S)
    assert len(kernels) == 2 * 4 * (2 + 2 + 1)
    for name, text in kernels:
        assert not _stores_before_restore(text.split("\n")), name
