"""Head norms with an eps below the smallest normal float32: a head of zeros has
x / sqrt(eps) * w = 0 for every eps > 0, and other heads of float16 values have a
mean square of 2^-57 at least (one element of 2^-24 among 512), beside which such
an eps is nothing. Bounds as in test_gpu_head_norms.
"""

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
from gpu_util import device, say
from test_gpu_head_norms import _check, _gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", (2.0 ** -126, 2.0 ** -127, 1e-40, 2.0 ** -149))
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 32), (512, 0)])
def test_zeros_stay_zeros(eps, D, rot):
    say(f"norm eps={eps} D={D}")
    rng = np.random.default_rng(D)
    x = rng.standard_normal((3, 2, D)).astype(np.float16)
    x[1] = 0
    x[2] = 0
    x[2, 0, 3] = 2.0 ** -24
    w = (1 + 0.3 * rng.standard_normal(D)).astype(np.float16)
    pos = np.array([3, 1, 2], np.int32)
    table = dq.rope_table(4, rot) if rot else None
    y = dq.rope(_gpu(x), _gpu(pos) if rot else None, table.to(device()) if rot else None, norm=_gpu(w), eps=eps)
    y = y.cpu().numpy()
    _check(y, x, w, pos, table.numpy() if rot else None, rot, False, eps=eps)
    assert not y[1].any() and not y[2, 1].any()
    if D <= 256 and D >= 64 and D & (D - 1) == 0:
        cache = dq.KVCache.empty(1, 2, D, 16, device=device())
        cache.k.fill_(7)
        slots = _gpu(np.arange(3, dtype=np.int32))
        q = dq.rope_append(cache, _gpu(x), _gpu(x), _gpu(x), _gpu(pos) if rot else None, slots,
                           table.to(device()) if rot else None, q_norm=_gpu(w), k_norm=_gpu(w), eps=eps)
        k = cache.k[0, :, :3].transpose(0, 1)
        for is_, name in ((q, "q"), (k, "k")):
            _check(is_.cpu().numpy(), x, w, pos, table.numpy() if rot else None, rot, False, eps=eps, what=name)


def test_zeros_without_eps_are_nan():
    """0 / 0, as the formula has it."""
    x = torch.zeros((1, 1, 64), dtype=torch.float16, device=device())
    assert torch.isnan(dq.rope(x, None, None, norm=torch.ones(64, dtype=torch.float16, device=device()), eps=0.0)).all()
