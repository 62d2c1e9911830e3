"""Token log probabilities at the largest vocabularies, where a row that starts
inside a 16-byte group is cut into one part more than an aligned one: for float32
more parts than the join has threads. What stands in the last part has to count.

Bounds: those of the other vocabularies (one addition more across parts).
"""

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
from gpu_util import device, say
from test_gpu_logprob import DTYPES, _check, _gpu

pytestmark = pytest.mark.gpu

MOST = 1 << 22


@pytest.mark.parametrize("V", (MOST - 4, MOST - 3, MOST - 2, MOST - 1, MOST))
@pytest.mark.parametrize("dtype", ("f16", "f32"))
@pytest.mark.parametrize("last", (1, 2))
def test_the_last_logits_count(V, dtype, last):
    """Contiguous rows of odd length, and rows one element behind a group's start; the largest logit among the last."""
    say(f"logprob longest V={V} {dtype} last={last}")
    rng = np.random.default_rng(V + last)
    x = (rng.standard_normal((2, V)) * 2).astype(DTYPES[dtype])
    x[:, V - last] = 25                     # as likely as all others together, and more
    tokens = np.array([V - last, 5], np.int32)
    _check(dq.token_logprobs(_gpu(x), _gpu(tokens), top=5), x, tokens, 5, "contiguous")
    wide = torch.zeros((2, V + 1), dtype=torch.float16 if dtype == "f16" else torch.float32, device=device())
    wide[:, 1:] = _gpu(x)
    _check(dq.token_logprobs(wide[:, 1:], _gpu(tokens), top=5), x, tokens, 5, "one element on")
    _check(dq.token_logprobs(wide[:1, 1:], _gpu(tokens[:1])), x[:1], tokens[:1], 0, "one row")
