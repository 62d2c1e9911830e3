"""The example decoder against a float64 model of it.

Tolerance: every operator rounds its result to float16 (relative 2^-11) and the
quantized products stay within a relative Frobenius error of 1e-3. Along the
residual stream two layers make 18 such steps and the head one; each adds at
most 1e-3 of its own result's norm, which the norms keep near that of the
stream, so that the logits are within 2e-2 relative Frobenius error. (A wrong
position, page, mask or order of heads is an error of about 1.) Quantized
caches are compared with a model that reads the values back from codes; the
codes differ where a value is within its own error of a rounding edge: a
fraction 2^-11 * 2^(bits - 1) of them, one code step each, which is below the
product's own error.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
import oracle
from gpu_util import device, say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("example_decoder", os.path.join(ROOT, "examples", "decoder.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


SHAPE = dict(layers=2, hidden=512, heads=8, kv_heads=2, mlp=768, vocab=512, pages=24, page_size=16, max_pos=256)


def _numbers(t):
    return t.double().cpu().numpy()


class Model:
    """The same decoder in float64, one sequence from its first token on."""

    def __init__(self, d, bits):
        self.d, self.bits = d, bits
        w = lambda m: _numbers(dq.dequant(m.layout, m.qweight, m.scales, None))      # noqa: E731
        self.layers = [{n: w(x[n]) for n in ("qkv", "out", "gate", "up", "down")} | {"norms": [_numbers(t) for t in x["norms"]]}
                       for x in d.layers]
        self.head, self.embedding, self.table = w(d.head), _numbers(d.embedding), _numbers(d.table)

    def cached(self, x):
        if self.bits == 16:
            return x
        c, s = oracle.kv_quantize(x.astype(np.float16).reshape(-1, self.d.dim), self.bits, 32)
        return oracle.kv_dequantize(c, s, self.d.dim, self.bits, 32).astype(np.float64).reshape(x.shape)

    def logits(self, tokens):
        d, T = self.d, len(tokens)
        H, Hk, D = d.heads, d.kv_heads, d.dim
        norm = lambda x, w: x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5) * w     # noqa: E731
        x = self.embedding[tokens]
        for w in self.layers:
            qkv = (norm(x, w["norms"][0]) @ w["qkv"]).reshape(T, H + 2 * Hk, D)
            q, k = (oracle.decoder.rope(t, np.arange(T), self.table, D, False) for t in (qkv[:, :H], qkv[:, H:H + Hk]))
            y, _, _ = oracle.decoder.attention(q, self.cached(k), self.cached(qkv[:, H + Hk:]), D ** -0.5, d.window)
            x = x + y.reshape(T, H * D) @ w["out"]
            y = norm(x, w["norms"][1])
            g = y @ w["gate"]
            x = x + (g / (1 + np.exp(-g)) * (y @ w["up"])) @ w["down"]
        return norm(x, 1.0) @ self.head


def _close(got, ref, what):
    rel = np.linalg.norm(_numbers(got) - ref) / np.linalg.norm(ref)
    assert rel <= 2e-2, f"{what}: relative error {rel:.2e}"


@pytest.mark.parametrize("bits,window", [(16, 0), (16, 20), (8, 0)])
def test_sequences_come_branch_and_go(bits, window):
    say(f"decoder example bits={bits} window={window}")
    device()
    d = _example().Decoder(bits=bits, window=window, seed=bits, **SHAPE)
    ref = Model(d, bits)
    tokens = np.random.default_rng(bits).integers(0, 512, 120).tolist()
    text = {"a": [], "b": [], "c": []}

    def step(*batch):
        got = d.step(list(batch))
        at = 0
        for seq, new in batch:
            text[seq] = text[seq] + new
            _close(got[at:at + len(new)], ref.logits(text[seq])[-len(new):], f"{seq} at {len(text[seq])}")
            at += len(new)

    d.add("a")
    step(("a", tokens[:37]))                                   # a prompt
    d.add("b")
    step(("a", tokens[37:38]), ("b", tokens[50:90]))           # a token, and another prompt
    d.fork("a", "c")                                           # inside a page: one copied, the rest shared
    text["c"] = list(text["a"])
    step(("c", [5]), ("a", [7]), ("b", tokens[90:95]))         # branches, and a draft of five
    d.pool.truncate("b", 42)                                   # three of them rejected
    text["b"] = text["b"][:42]
    step(("a", [1]), ("b", [2]), ("c", [3]))
    d.free("a")
    d.compact()
    step(("c", tokens[100:120]), ("b", [9]))
    step(("b", [11]), ("c", [12]))
    d.free("b")
    d.free("c")
    assert d.pool.free_pages == SHAPE["pages"]


def test_captured_step():
    """The forward pass of single tokens in a graph: replayed with new
    positions, slots and lengths in place, equal to the eager call."""
    say("decoder example graph")
    dev = device()
    d = _example().Decoder(seed=3, **SHAPE)
    d.add("a")
    d.add("b")
    d.step([("a", list(range(40))), ("b", list(range(9)))])
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
    tokens, positions, slots, lens = ints([1, 2]), ints([0, 0]), ints([-1, -1]), ints([1, 1])
    where = dict(block_table=torch.zeros((2, 4), dtype=torch.int32, device=dev), kv_len=lens, q_start=ints([0, 1, 2]),
                 max_q_len=1, max_kv_len=64, window=0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.forward(tokens, positions, slots, where)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = d.forward(tokens, positions, slots, where)
    for i in range(12):
        at = [d.pool.length(s) for s in "ab"]
        slots.copy_(ints([d.pool.extend(s, 1)[0] for s in "ab"]))
        positions.copy_(ints(at))
        lens.copy_(ints([n + 1 for n in at]))
        tokens.copy_(ints([i, 100 + i]))
        where["block_table"].copy_(ints([(d.pool.pages(s) + [0] * 4)[:4] for s in "ab"]))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = d.forward(tokens, positions, slots, where)
        torch.cuda.synchronize()
        assert torch.isfinite(got).all() and torch.equal(got, eager), i
