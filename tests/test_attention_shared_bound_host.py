"""What the bound of the shared lengths decides on: nothing but its own check. No GPU needed."""

import ctypes

import pytest

import dequant_matmul_gptq_amd as dq
from test_attention_views_host import INV, TOP, _cache


@pytest.mark.parametrize("sizes", [(3, 8, 2, 3, 100, 1), (32, 64, 32, 1, 17000, 1), (600, 16, 20, 300, 9000, 4)])
@pytest.mark.parametrize("bits", (16, 4))
def test_the_workspace_does_not_depend_on_it(sizes, bits):
    f, c = dq.lib().qlinear_paged_attention_shared_workspace_bytes, _cache(bits=bits)
    need = []
    for most in (0, 1, sizes[4], TOP):
        n = ctypes.c_size_t(0)
        assert f(ctypes.byref(c), *sizes, most, ctypes.byref(n)) == 0
        need.append(n.value)
    assert need[0] > 0 and len(set(need)) == 1
    assert f(ctypes.byref(c), *sizes, -1, ctypes.byref(n)) == INV
