"""The example decoder with normed heads, sinks, branches that read their shared
pages once, and log probabilities: the operators together, against a float64
model of it.

Tolerance: that of the decoder without them (every operator rounds its result to
float16; two layers and the head keep the logits within 2e-2 relative Frobenius
error). The norms of heads add two such roundings a layer; a norm, mask, group or
row of the wrong head or sequence is an error of about 1. Log probabilities are
taken of the same float16 logits in 64 bits: |x| up to 16 with sums of 512 terms
in float32 leave 16 * 2^-24 for the largest, the sum's 512 * 2^-24 / 2 and the
logarithm's own 4 * 2^-24: below 2e-5.
"""

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
import oracle
from gpu_util import device, say
from test_gpu_decoder_example import SHAPE, Model, _close, _example, _numbers

pytestmark = pytest.mark.gpu


class ViewModel(Model):
    def __init__(self, d, bits):
        super().__init__(d, bits)
        self.head_norms = [[None if w is None else _numbers(w) for w in x["head_norms"]] for x in d.layers]

    def logits(self, tokens):
        d, T = self.d, len(tokens)
        H, Hk, D = d.heads, d.kv_heads, d.dim
        norm = lambda x, w, eps=1e-5: x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w     # noqa: E731
        x = self.embedding[tokens]
        for w, head_norms in zip(self.layers, self.head_norms):
            qkv = (norm(x, w["norms"][0]) @ w["qkv"]).reshape(T, H + 2 * Hk, D)
            q, k = (t if n is None else norm(t, n, 1e-6) for t, n in zip((qkv[:, :H], qkv[:, H:H + Hk]), head_norms))
            q, k = (oracle.decoder.rope(t, np.arange(T), self.table, D, False) for t in (q, k))
            y, _, _ = oracle.decoder.attention(q, self.cached(k), self.cached(qkv[:, H + Hk:]), D ** -0.5, d.window,
                                               sinks=d.sinks)
            x = x + y.reshape(T, H * D) @ w["out"]
            y = norm(x, w["norms"][1])
            g = y @ w["gate"]
            x = x + (g / (1 + np.exp(-g)) * (y @ w["up"])) @ w["down"]
        return norm(x, 1.0) @ self.head


@pytest.mark.parametrize("bits,window,sinks,head_norms", [(16, 0, 0, True), (16, 20, 5, False), (8, 0, 0, False),
                                                          (8, 20, 17, True), (4, 0, 0, True)])
def test_branches_with_all_of_it(bits, window, sinks, head_norms):
    say(f"decoder example bits={bits} window={window} sinks={sinks} head norms={head_norms}")
    dev = device()
    d = _example().Decoder(bits=bits, window=window, sinks=sinks, head_norms=head_norms, share=True, seed=bits, **SHAPE)
    ref = ViewModel(d, bits)
    tokens = np.random.default_rng(bits + 1).integers(0, 512, 160).tolist()
    text, groups = {}, []
    forward = d.forward

    def watched(*args):
        groups.append("shared_len" in args[3] and args[3]["shared_len"].tolist())
        return forward(*args)

    d.forward = watched

    def step(*batch):
        got = d.step(list(batch))
        at = 0
        for seq, new in batch:
            text[seq] = text.get(seq, []) + new
            _close(got[at:at + len(new)], ref.logits(text[seq])[-len(new):], f"{seq} at {len(text[seq])}")
            at += len(new)
        asked = torch.tensor([n for _, new in batch for n in new], dtype=torch.int32, device=dev)
        r = dq.token_logprobs(got, asked, top=7)
        x = _numbers(got)
        x = x - x.max(1, keepdims=True)
        lp = x - np.log(np.exp(x).sum(1, keepdims=True))
        order = np.argsort(-lp, axis=1, kind="stable")[:, :7]
        assert np.array_equal(r.top_id.cpu().numpy(), order)
        for name, is_, want in (("logprob", r.logprob, np.take_along_axis(lp, asked.cpu().numpy()[:, None], 1)[:, 0]),
                                ("top", r.top_logprob, np.take_along_axis(lp, order, 1)),
                                ("entropy", r.entropy, -(np.exp(lp) * lp).sum(1))):
            assert np.abs(_numbers(is_) - want).max() <= 2e-5, name
        return got

    d.add("a")
    step(("a", tokens[:50]))                                   # three whole pages and two tokens
    for name in "bc":
        d.fork("a", name)
        text[name] = list(text["a"])
    d.add("x")
    step(("a", [3]), ("b", [7, 8, 9]), ("c", [1]), ("x", tokens[60:90]))      # branches, and another prompt
    d.fork("x", "y")
    text["y"] = list(text["x"])
    step(("a", [5]), ("b", [6]), ("c", tokens[90:100]), ("x", [2]), ("y", [4]))
    d.free("a")
    d.compact()
    step(("y", [11]), ("x", [12]), ("c", [13]), ("b", [14, 15]))
    want = [False, [48, 0], [48, 16], [16, 48]] if window == 0 else [False] * 4
    assert groups == want
