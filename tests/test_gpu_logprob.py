"""Log probabilities of given tokens, entropy and top alternatives against the
float64 oracle.

Bounds. A term's exponent t = x log2 e - c has a relative error of 2^-23 (one
fused multiply-add, log2 e rounded), the exponential 2^-23, and a sum up to 128
additions in a thread, 16 across threads and waves and 16 across parts, each
2^-24: log l is off by 160 * 2^-24 and 2^-22 times the terms' mean |t| at most
(below 2^-22 |m - x| of the furthest term that counts, 24 ln 2 for what stays
above 2^-24 of the largest; terms further down add less than V 2^-24 of it each).
A log probability adds its own t's error, 2^-22 |log p|, and its rounding:
  |err| <= 2^-16 + 2^-21 |log p|
The entropy's second sum has the same relative error of its terms |p log2 p|,
whose sum is H + log l at most:  |err| <= 2^-16 (1 + 2 (H + ln V)).
The top indexes are compared with the order itself.
"""

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
import oracle
from gpu_util import Guarded, device, say

pytestmark = pytest.mark.gpu

DTYPES = {"f16": np.float16, "f32": np.float32}


def _gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device())


def _check(r, x, tokens, top, what=""):
    lp, h = oracle.decoder.log_probabilities(x)
    rows = np.arange(x.shape[0])

    def close(got, want, bound, name):
        got, fine = got.cpu().numpy().astype(np.float64), np.isfinite(want)
        assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what} {name}: NaN"
        assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{what} {name}: infinities"
        err = np.abs(got[fine] - want[fine])
        assert (err <= bound[fine]).all(), f"{what} {name}: {err.max():.3e}, {(err / bound[fine]).max():.2f} bounds"

    if tokens is not None:
        inside = (tokens >= 0) & (tokens < x.shape[1])
        want = np.where(inside, lp[rows, np.where(inside, tokens, 0)], np.nan)
        with np.errstate(invalid="ignore"):
            close(r.logprob, want, 2.0 ** -16 + 2.0 ** -21 * np.abs(want), "logprob")
    if r.entropy is not None:
        close(r.entropy, h, 2.0 ** -16 * (1 + 2 * (h + np.log(x.shape[1]))), "entropy")
    if top:
        ids = oracle.decoder.top_indexes(x, top)
        assert np.array_equal(r.top_id.cpu().numpy(), ids), f"{what}: top"
        want = np.take_along_axis(lp, ids, 1)
        with np.errstate(invalid="ignore"):
            close(r.top_logprob, want, 2.0 ** -16 + 2.0 ** -21 * np.abs(want), "top logprob")
    else:
        assert r.top_id is None and r.top_logprob is None


def _logits(rng, R, V, dtype):
    x = rng.standard_normal((R, V)) * 3
    x[::2, V // 2] += 12
    return x.astype(DTYPES[dtype])


@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 63, 64, 65, 100, 255, 1000, 2047, 2048, 2049, 4097])
@pytest.mark.parametrize("dtype", ("f16", "f32"))
def test_small_vocabularies(V, dtype):
    say(f"logprob V={V} {dtype}")
    rng = np.random.default_rng(V)
    for R in (1, 6):
        x, tokens = _logits(rng, R, V, dtype), rng.integers(0, V, R).astype(np.int32)
        for top in sorted({0, 1, min(2, V), min(V, 5), min(V, 64)}):
            _check(dq.token_logprobs(_gpu(x), _gpu(tokens), top=top), x, tokens, top, f"R={R} top={top}")


@pytest.mark.parametrize("R,V", [(1, 32000), (1, 131072), (2, 32001), (5, 50001), (64, 32000), (600, 4096), (600, 33001),
                                 (130, 70001), (1, 1000003)])
@pytest.mark.parametrize("dtype", ("f16", "f32"))
@pytest.mark.parametrize("top", (0, 1, 20, 64))
def test_vocabularies(R, V, dtype, top):
    say(f"logprob R={R} V={V} {dtype} top={top}")
    rng = np.random.default_rng(R + V)
    x, tokens = _logits(rng, R, V, dtype), rng.integers(0, V, R).astype(np.int32)
    _check(dq.token_logprobs(_gpu(x), _gpu(tokens), top=top), x, tokens, top)


@pytest.mark.parametrize("R,V", [(3, 1000), (2, 5000), (2, 40000), (300, 20000)])
@pytest.mark.parametrize("dtype", ("f16", "f32"))
def test_rows_in_order_and_equal_rows(R, V, dtype):
    """Orders that put the largest in few threads, and more equal elements than are ranked at once."""
    say(f"logprob order R={R} V={V} {dtype}")
    up = np.linspace(-8, 8, V)
    few = np.where(np.arange(V) % 997 < 3, 2.0, -1.0)
    block = np.where((np.arange(V) >= V // 3) & (np.arange(V) < V // 3 + 700), 4.0, 0.0)
    zeros = np.where(np.arange(V) % 2 == 0, 0.0, -0.0)
    for name, row in (("up", up), ("down", up[::-1]), ("equal", np.full(V, 1.5)), ("few", few), ("block", block),
                      ("zeros", zeros), ("one", np.where(np.arange(V) == V - 1, 30.0, -30.0))):
        x = np.broadcast_to(row, (R, V)).astype(DTYPES[dtype])
        tokens = np.arange(R).astype(np.int32)
        for top in (1, 5, 64):
            _check(dq.token_logprobs(_gpu(x), _gpu(tokens), top=top), x, tokens, top, f"{name} top={top}")


@pytest.mark.parametrize("V", (70, 3000, 40001))
@pytest.mark.parametrize("dtype", ("f16", "f32"))
def test_masks_infinities_and_nan(V, dtype):
    say(f"logprob masks V={V} {dtype}")
    rng = np.random.default_rng(V)
    for R in (9, 400):
        x = _logits(rng, R, V, dtype)
        x[0, rng.random(V) < 0.7] = -np.inf
        x[1] = -np.inf                       # nothing can come
        x[2] = -np.inf
        x[2, V - 3] = -5                     # one token can
        x[3] = np.finfo(x.dtype).min         # a mask of the lowest value
        x[3, 7] = 1
        x[4] = np.finfo(x.dtype).min         # and nothing else
        x[5, 11] = np.nan
        x[6, 12] = np.inf
        x[7, [3, 40, V - 1]] = np.nan
        x[8] = np.nan
        tokens = np.full(R, 7, np.int32)
        tokens[2] = V - 3
        for top in (0, 1, 5, 64):
            _check(dq.token_logprobs(_gpu(x), _gpu(tokens), top=top), x, tokens, top, f"R={R} top={top}")


def test_tokens_outside_the_vocabulary_give_nan():
    say("logprob tokens")
    rng = np.random.default_rng(3)
    x = _logits(rng, 6, 500, "f16")
    tokens = np.array([0, -1, 499, 500, 2 ** 31 - 1, -2 ** 31], np.int32)
    r = dq.token_logprobs(_gpu(x), _gpu(tokens), top=2)
    _check(r, x, tokens, 2)
    assert np.isnan(r.logprob.cpu().numpy()).tolist() == [False, True, False, True, True, True]


@pytest.mark.parametrize("dtype", ("f16", "f32"))
@pytest.mark.parametrize("R,V,wide,at", [(5, 1000, 1003, 1), (3, 32000, 32007, 3), (300, 4001, 4001, 0), (7, 17, 33, 5),
                                         (4, 9, 12, 2)])
def test_strides_and_alignment(dtype, R, V, wide, at):
    """Rows that start anywhere, in a buffer whose other elements are larger than all of theirs."""
    say(f"logprob strides R={R} V={V} {dtype}")
    rng = np.random.default_rng(V + at)
    x, tokens = _logits(rng, R, V, dtype), rng.integers(0, V, R).astype(np.int32)
    raw = np.full((R, wide), 1000, DTYPES[dtype])
    raw[:, at:at + V] = x
    top = min(V, 20)
    size = x.dtype.itemsize
    g = Guarded(R * wide * size, device())
    buf = g.view(torch.float16 if size == 2 else torch.float32, (R, wide))
    buf.copy_(_gpu(raw))
    _check(dq.token_logprobs(buf[:, at:at + V], _gpu(tokens), top=top), x, tokens, top)
    assert g.intact()


def test_outputs_stay_inside_and_each_may_be_left_out():
    say("logprob outputs")
    rng = np.random.default_rng(4)
    for R, V, top in ((3, 40000, 20), (700, 900, 3)):
        x, tokens = _logits(rng, R, V, "f16"), rng.integers(0, V, R).astype(np.int32)
        guards = [Guarded(4 * n, device()) for n in (R, R, R * top, R * top)]
        views = [g.view(t, s) for g, t, s in zip(guards, (torch.float32,) * 3 + (torch.int32,), ((R,), (R,), (R, top), (R, top)))]
        ws = Guarded(dq.token_logprobs_workspace_bytes(R, V, top) or 16, device())
        r = dq.token_logprobs(_gpu(x), _gpu(tokens), top=top, out=dq.TokenLogprobs(*views),
                              workspace=ws.bytes())
        assert all(g.intact() for g in guards) and ws.intact()
        _check(r, x, tokens, top)
        r = dq.token_logprobs(_gpu(x), top=top, entropy=False)
        assert r.logprob is None and r.entropy is None and torch.equal(r.top_id, views[3])
        r = dq.token_logprobs(_gpu(x), _gpu(tokens), entropy=False)
        assert torch.equal(r.logprob, views[0]) and r.entropy is None and r.top_id is None
        assert all(t is None for t in dq.token_logprobs(_gpu(x), entropy=False))
    r = dq.token_logprobs(torch.empty((0, 50), dtype=torch.float16, device=device()), top=3)
    assert r.entropy.shape == (0,) and r.top_id.shape == (0, 3)


def test_one_workspace_for_smaller_calls():
    say("logprob workspace")
    rng = np.random.default_rng(8)
    ws = dq.token_logprobs_workspace(64, 70000, 20)
    for R, V, top in ((64, 70000, 20), (1, 70000, 20), (17, 32000, 5), (64, 3000, 1), (3, 69999, 0)):
        x, tokens = _logits(rng, R, V, "f16"), rng.integers(0, V, R).astype(np.int32)
        _check(dq.token_logprobs(_gpu(x), _gpu(tokens), top=top, workspace=ws), x, tokens, top)


def test_results_do_not_change_from_call_to_call():
    say("logprob repeat")
    rng = np.random.default_rng(9)
    x = _gpu(_logits(rng, 40, 32000, "f16"))
    tokens = _gpu(rng.integers(0, 32000, 40).astype(np.int32))
    a = dq.token_logprobs(x, tokens, top=20)
    for _ in range(3):
        b = dq.token_logprobs(x, tokens, top=20)
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_logprobs_in_a_graph_and_on_another_stream():
    say("logprob graph")
    rng = np.random.default_rng(10)
    x, tokens = _gpu(_logits(rng, 4, 32000, "f16")), _gpu(np.array([5, 6, 7, 8], np.int32))
    ws = dq.token_logprobs_workspace(4, 32000, 5)
    out = dq.token_logprobs(x, tokens, top=5, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dq.token_logprobs(x, tokens, top=5, out=out, workspace=ws)
    for _ in range(3):
        x.copy_(_gpu(_logits(rng, 4, 32000, "f16")))
        graph.replay()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            want = dq.token_logprobs(x, tokens, top=5)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
