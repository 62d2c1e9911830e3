"""Host-side tests of the head norms and the log probabilities: refusals of the
C entry points (made before any launch) and of the binding, workspace queries,
and pins of the oracle's functions. No GPU needed."""

import ctypes
import math
import os
import random
import shutil
import subprocess

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
from dequant_matmul_gptq_amd import _lib
from oracle import decoder_oracle as od

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000      # never dereferenced: every call here is refused first
INV, UNS, MIS, WSP = (_lib.ERR_INVALID_ARGUMENT, _lib.ERR_UNSUPPORTED, _lib.ERR_MISALIGNED, _lib.ERR_WORKSPACE)


def _cache(**kw):
    f = dict(k=FAKE, v=FAKE, k_scales=FAKE, v_scales=FAKE, num_pages=4, page_size=32, kv_heads=2, head_dim=128,
             bits=16, group=32)
    f.update(kw)
    return _lib.qlinear_kv_cache(*[f[n] for n, _ in _lib.qlinear_kv_cache._fields_])


# ---------------------------------------------------------------- head norms

ROPE = dict(x=FAKE, x_stride=256, tokens=2, heads=2, head_dim=128, weight=FAKE, weight_heads=1, eps=1e-6,
            positions=FAKE, table=FAKE, table_rows=9, rot_dim=64, layout=0, out=FAKE, out_stride=256)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INV), (dict(out=None), INV), (dict(positions=None), INV), (dict(table=None), INV),
    (dict(weight=None), INV), (dict(weight_heads=3), INV), (dict(weight_heads=0), INV), (dict(eps=-1e-6), INV),
    (dict(eps=math.nan), INV), (dict(eps=math.inf), INV), (dict(tokens=-1), INV), (dict(heads=-1), INV),
    (dict(head_dim=0), INV), (dict(rot_dim=-16), INV), (dict(table_rows=0), INV), (dict(x_stride=248), INV),
    (dict(x_stride=260), UNS), (dict(head_dim=120), UNS), (dict(rot_dim=24), UNS), (dict(rot_dim=144), UNS),
    (dict(layout=2), UNS), (dict(head_dim=528, x_stride=2048, out_stride=2048), UNS), (dict(heads=65536), UNS),
    (dict(tokens=1 << 22), UNS), (dict(x=FAKE + 8), MIS), (dict(weight=FAKE + 8), MIS), (dict(table=FAKE + 8), MIS)])
def test_norm_rope_refuses(change, status):
    a = dict(ROPE)
    a.update(change)
    assert dq.lib().qlinear_norm_rope(*a.values(), None) == status


def test_norm_rope_no_work():
    for change in (dict(tokens=0), dict(heads=0)):
        a = dict(ROPE, x=None, weight=None, out=None, positions=None, table=None)
        a.update(change)
        assert dq.lib().qlinear_norm_rope(*a.values(), None) == 0


APPEND = dict(q=FAKE, q_stride=1024, q_heads=8, k=FAKE, k_stride=256, v=FAKE, v_stride=256, q_out=FAKE,
              q_out_stride=1024, tokens=1, q_norm=FAKE, q_norm_heads=1, k_norm=FAKE, k_norm_heads=2, eps=1e-6,
              positions=FAKE, slots=FAKE, table=FAKE, table_rows=8, rot_dim=64, layout=0)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(slots=None), INV), (dict(q_out=None), INV),
    (dict(q_norm_heads=2), INV), (dict(k_norm_heads=8), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV),
    (dict(tokens=-1), INV), (dict(q_heads=-1), INV), (dict(rot_dim=-1), INV), (dict(rot_dim=8), UNS),
    (dict(tokens=1 << 22), UNS), (dict(q_heads=65536), UNS), (dict(q_norm=FAKE + 2), MIS), (dict(k_norm=FAKE + 8), MIS),
    (dict(slots=FAKE + 2), MIS), (dict(k=FAKE + 8), MIS)])
def test_norm_rope_append_refuses(change, status):
    a = dict(APPEND)
    a.update(change)
    c = _cache()
    assert dq.lib().qlinear_norm_rope_append(ctypes.byref(c), *a.values(), None) == status


def test_norm_rope_append_checks_the_cache():
    f = dq.lib().qlinear_norm_rope_append
    assert f(None, *APPEND.values(), None) == INV
    for change, status in ((dict(k=None), INV), (dict(page_size=48), UNS), (dict(bits=8, group=16), UNS), (dict(v=FAKE + 8), MIS)):
        assert f(ctypes.byref(_cache(**change)), *APPEND.values(), None) == status
    assert f(ctypes.byref(_cache()), *dict(APPEND, tokens=0, q=None, k=None, v=None).values(), None) == 0


# ---------------------------------------------------------------- log probabilities

LOGPROB = dict(logits=FAKE, stride=1000, rows=3, vocab=1000, logit_bits=16, tokens=FAKE, top=5, logprob=FAKE,
               entropy=FAKE, top_logprob=FAKE, top_id=FAKE, workspace=FAKE, workspace_bytes=1 << 30)


def _logprob(**kw):
    return dq.lib().qlinear_token_logprobs(*dict(LOGPROB, **kw).values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), INV), (dict(tokens=None), INV), (dict(top_logprob=None), INV), (dict(top_id=None), INV),
    (dict(rows=-1), INV), (dict(vocab=0), INV), (dict(top=-1), INV), (dict(top=1001), INV), (dict(stride=999), INV),
    (dict(vocab=4, top=5, stride=8), INV), (dict(logit_bits=8), UNS), (dict(logit_bits=64), UNS), (dict(top=65), UNS),
    (dict(vocab=(1 << 22) + 1, stride=1 << 23), UNS), (dict(rows=1 << 22), UNS),
    (dict(rows=(1 << 15) + 1, vocab=1 << 22, stride=1 << 22), UNS), (dict(logits=FAKE + 1), MIS),
    (dict(logits=FAKE + 2, logit_bits=32), MIS), (dict(tokens=FAKE + 2), MIS), (dict(logprob=FAKE + 1), MIS),
    (dict(entropy=FAKE + 2), MIS), (dict(top_logprob=FAKE + 2), MIS), (dict(top_id=FAKE + 1), MIS)])
def test_logprob_refuses(change, status):
    assert _logprob(**change) == status


def test_logprob_no_work_and_workspace():
    assert _logprob(rows=0, logits=None, tokens=None) == 0
    assert _logprob(logprob=None, entropy=None, top=0) == 0
    f, n = dq.lib().qlinear_token_logprobs_workspace_bytes, ctypes.c_size_t(77)
    assert f(3, 1000, 16, 5, None) == INV
    assert f(0, 1000, 16, 5, ctypes.byref(n)) == 0 and n.value == 0
    for sizes, status in (((-1, 1000, 16, 5), INV), ((3, 0, 16, 5), INV), ((3, 1000, 12, 5), UNS), ((3, 1000, 16, 65), UNS),
                          ((3, 4, 16, 5), INV)):
        assert f(*sizes, ctypes.byref(n)) == status
    # one long row is cut: it needs a workspace, and says so
    assert f(1, 100000, 16, 5, ctypes.byref(n)) == 0 and n.value > 0
    long = dict(rows=1, vocab=100000, stride=100000)
    assert _logprob(workspace=None, **long) == WSP
    assert _logprob(workspace_bytes=100, **long) == WSP
    assert _logprob(workspace=FAKE + 8, **long) == MIS
    with pytest.raises(dq.QlinearError) as e:
        dq.token_logprobs_workspace_bytes(2 ** 32 + 1, 1000)
    assert e.value.status == UNS


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    exe = str(tmp_path_factory.mktemp("probe") / "logprob_probe")
    cmd = [hipcc, "-std=c++20", "-O1", "-x", "hip", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "dequant_matmul_gptq_amd", "csrc"),
           os.path.join(ROOT, "tests", "host", "logprob_probe.cpp"), "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]

    return run


@pytest.mark.parametrize("seed", range(3))
def test_a_logprob_workspace_covers_smaller_calls(ask, seed):
    rng = random.Random(seed)
    log = lambda hi: int(hi ** rng.random() + 0.5)      # noqa: E731
    for _ in range(20):
        bits, most = rng.choice((16, 32)), (log(5000), log(1 << 22), rng.randrange(65))
        cases = [(*most[:2], bits, most[2])]
        for _ in range(300):
            rows, vocab = (rng.choice((log(x), x, max(1, x - rng.randrange(40)))) for x in most[:2])
            cases.append((rows, vocab, bits, rng.randrange(most[2] + 1)))
        got = ask(cases)
        assert len(got) == len(cases)
        for case, (need, _) in zip(cases, got):
            assert need <= got[0][1], (cases[0], case)


# ---------------------------------------------------------------- binding and oracle

def test_binding_refuses_host_tensors():
    x, w = torch.zeros((4, 2, 64), dtype=torch.float16), torch.ones(64, dtype=torch.float16)
    for call in (lambda: dq.rope(x, None, None, norm=w), lambda: dq.token_logprobs(x[0]),
                 lambda: dq.token_logprobs(torch.zeros((3, 8)), torch.zeros(3, dtype=torch.int32), top=2)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_oracle_head_norm_and_logprob_pins():
    y = od.head_norm(np.array([[[3.0, 4.0], [6.0, 8.0]]]), np.array([1.0, 2.0]), 0.0)
    r = math.sqrt(12.5)
    assert np.allclose(y, [[[3 / r, 8 / r], [3 / r, 8 / r]]])
    y = od.head_norm(np.array([[[3.0, 4.0], [6.0, 8.0]]]), np.array([[1.0, 2.0], [0.0, 1.0]]), 0.0)
    assert np.allclose(y, [[[3 / r, 8 / r], [0, 4 / r]]])
    inf = math.inf
    lp, h = od.log_probabilities([[0.0, math.log(3.0), -inf], [5.0, 5.0, 5.0], [-inf, -inf, -inf], [0, inf, 0], [0, math.nan, 1]])
    assert np.allclose(lp[0], [math.log(0.25), math.log(0.75), -inf])
    assert np.isclose(h[0], -0.25 * math.log(0.25) - 0.75 * math.log(0.75))
    assert np.allclose(lp[1], -math.log(3)) and np.isclose(h[1], math.log(3))
    assert np.isnan(lp[2:]).all() and np.isnan(h[2:]).all()
    assert od.top_indexes([[1, 3, 3, 2], [0.0, -0.0, -1, math.nan], [-inf, -inf, -inf, 0]], 3).tolist() == \
        [[1, 2, 3], [3, 0, 1], [3, 0, 1]]


def test_oracle_attention_with_sinks_pins():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((9, 1, 4))
    ones = np.ones((9, 1, 4))
    o, _, total = od.attention(np.ones((2, 1, 4)), ones, v, 0.3, window=3, sinks=2)
    assert np.allclose(o[0, 0], v[[0, 1, 5, 6, 7], 0].mean(0)) and np.allclose(o[1, 0], v[[0, 1, 6, 7, 8], 0].mean(0))
    assert np.allclose(total, 5)
    # sinks inside the window are seen once
    o, _, total = od.attention(np.ones((1, 1, 4)), ones[:4], v[:4], 0.3, window=3, sinks=3)
    assert np.allclose(o[0, 0], v[:4, 0].mean(0)) and np.allclose(total, 4)
    o, _, total = od.attention(np.ones((1, 1, 4)), ones, v, 0.3, sinks=5)
    assert np.allclose(total, 9)
