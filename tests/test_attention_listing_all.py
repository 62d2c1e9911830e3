"""The two checks of the built attention kernels, for the instances that the others
leave out: registers stored to scratch memory while lanes are off
(test_attention_listing_views looks over the views' few-row kernels) in all other
kernels of the attention and in those of the rotary step and the log
probabilities, and the waits for rows on their way to LDS (test_attention_listing
follows the plain prompt kernels) in the views' prompt kernels. No GPU needed, but
the compiler."""

import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from dequant_matmul_gptq_amd import build
from test_attention_listing import _unwaited
from test_attention_listing_views import _stores_before_restore

# Kernels of each source.
FEW = {"attention_few_64.hip": 16, "attention_few_128.hip": 16, "attention_few_256.hip": 8}
CHUNK = {f"attention_{view}chunk_{d}.hip": 4 for view in ("", "view_") for d in (64, 128, 256)}
OTHERS = {"attention_views.hip": 9, "paged_attention.hip": 12, "logprob.hip": 12, "rope.hip": 176}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Lines of every kernel by its name, by source."""
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
            return {k: text.split("\n") for k, text in
                    re.findall(r"^(_Z\w*kernel\w*):(.*?)^\.Lfunc_end", f.read(), re.M | re.S)}

    names = [*FEW, *CHUNK, *OTHERS]
    with cf.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as ex:
        return dict(zip(names, ex.map(make, names)))


@pytest.mark.parametrize("source,count", [*FEW.items(), *CHUNK.items(), *OTHERS.items()])
def test_no_register_is_stored_while_lanes_are_off(kernels, source, count):
    assert len(kernels[source]) == count
    for name, lines in kernels[source].items():
        assert not _stores_before_restore(lines), name


@pytest.mark.parametrize("source", [s for s in CHUNK if "view" in s])
def test_views_wait_for_their_rows_before_the_barrier(kernels, source):
    found = {name: _unwaited(lines) for name, lines in kernels[source].items()}
    assert all(not bad for bad, _ in found.values()), found
    assert sorted(loads > 0 for _, loads in found.values()) == [False, False, False, True]      # codes go through registers
