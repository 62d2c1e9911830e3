"""Host-side tests of attention with sinks and over shared prefixes: refusals of
the C entry points (made before any launch) and of the binding, the workspace,
rows and lengths of groups, and the page pool's count of shared tokens. The
launch code is compiled for the host; no GPU needed."""

import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest
import torch

import dequant_matmul_gptq_amd as dq
from dequant_matmul_gptq_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000      # never dereferenced: every call here is refused first
INV, UNS, MIS, WSP = (_lib.ERR_INVALID_ARGUMENT, _lib.ERR_UNSUPPORTED, _lib.ERR_MISALIGNED, _lib.ERR_WORKSPACE)
TOP = 2 ** 31 - 1


def _cache(**kw):
    f = dict(k=FAKE, v=FAKE, k_scales=FAKE, v_scales=FAKE, num_pages=4, page_size=32, kv_heads=2, head_dim=128,
             bits=16, group=32)
    f.update(kw)
    return _lib.qlinear_kv_cache(*[f[n] for n, _ in _lib.qlinear_kv_cache._fields_])


SINKS = dict(q=FAKE, q_stride=1024, tokens=3, q_heads=8, batch=1, q_start=FAKE, kv_len=FAKE, block_table=FAKE,
             table_width=4, max_q_len=3, max_kv_len=100, scale=0.1, window=40, sinks=4, out=FAKE, ws=FAKE,
             ws_bytes=1 << 30)
SHARED = dict(q=FAKE, q_stride=1024, tokens=3, q_heads=8, batch=2, q_start=FAKE, kv_len=FAKE, block_table=FAKE,
              table_width=4, groups=1, shared_start=FAKE, shared_len=FAKE, max_q_len=3, max_kv_len=100,
              max_shared_len=64, scale=0.1, out=FAKE, ws=FAKE, ws_bytes=1 << 30)


def _sinks(cache=None, **kw):
    return dq.lib().qlinear_paged_attention_sinks(ctypes.byref(cache or _cache()), *dict(SINKS, **kw).values(), None)


def _shared(cache=None, **kw):
    return dq.lib().qlinear_paged_attention_shared(ctypes.byref(cache or _cache()), *dict(SHARED, **kw).values(), None)


BOTH = [(dict(q=None), INV), (dict(kv_len=None), INV), (dict(block_table=None), INV), (dict(out=None), INV),
        (dict(tokens=-1), INV), (dict(q_heads=0), INV), (dict(batch=-1), INV), (dict(table_width=0), INV),
        (dict(max_q_len=-1), INV), (dict(max_kv_len=-1), INV), (dict(scale=math.inf), INV), (dict(scale=math.nan), INV),
        (dict(q_start=None, batch=2), INV), (dict(q_stride=1016), INV), (dict(q_stride=1028), UNS),
        (dict(q_heads=7, q_stride=2048), UNS), (dict(batch=65536), UNS), (dict(tokens=1 << 30), UNS),
        (dict(q=FAKE + 2), MIS), (dict(out=FAKE + 4), MIS), (dict(kv_len=FAKE + 1), MIS), (dict(q_start=FAKE + 2), MIS),
        (dict(block_table=FAKE + 2), MIS)]


@pytest.mark.parametrize("change,status", BOTH + [(dict(window=-1), INV), (dict(sinks=-1), INV)])
def test_sinks_refuse(change, status):
    assert _sinks(**change) == status


@pytest.mark.parametrize("change,status", BOTH + [
    (dict(groups=0), INV), (dict(groups=-1), INV), (dict(shared_len=None), INV), (dict(groups=2, shared_start=None), INV),
    (dict(max_shared_len=-1), INV), (dict(shared_len=FAKE + 2), MIS), (dict(shared_start=FAKE + 1), MIS),
    (dict(batch=65000, groups=600), UNS), (dict(tokens=(1 << 22) + 1), UNS), (dict(batch=8000, groups=200, table_width=32768), UNS)])
def test_shared_refuses(change, status):
    assert _shared(**change) == status


def test_views_refuse_what_their_indexes_cannot_hold():
    for call in (_sinks, _shared):
        assert call(cache=_cache(kv_heads=4097), q_heads=4097, q_stride=4097 * 128) == UNS
        assert call(cache=_cache(kv_heads=128), q_heads=128, q_stride=128 * 128, batch=32769) == UNS
        assert call(batch=8193, table_width=32768) == UNS
        for change, status in ((dict(k=None), INV), (dict(page_size=48), UNS), (dict(bits=8, group=16), UNS), (dict(v=FAKE + 8), MIS)):
            assert call(cache=_cache(**change)) == status


def test_views_no_work_and_workspace_query():
    L, c = dq.lib(), _cache()
    for call in (_sinks, _shared):
        assert call(tokens=0, q=None, out=None) == 0 and call(batch=0, q=None, out=None) == 0
    n = ctypes.c_size_t(77)
    f = L.qlinear_paged_attention_sinks_workspace_bytes
    assert f(ctypes.byref(c), 1, 8, 1, 1, 1, 4, 0, None) == INV
    assert f(ctypes.byref(c), 1, 8, 1, 1, 1, 4, -1, ctypes.byref(n)) == INV
    assert f(ctypes.byref(c), 0, 8, 0, 0, 0, 0, 4, ctypes.byref(n)) == 0 and n.value == 0
    assert f(ctypes.byref(c), 1, 8, 1, 1, 100000, 5000, 4, ctypes.byref(n)) == 0 and n.value > 0
    long = dict(tokens=1, max_q_len=1, max_kv_len=100000, window=5000, table_width=4000)
    assert _sinks(ws=None, **long) == WSP and _sinks(ws_bytes=1000, **long) == WSP and _sinks(ws=FAKE + 8, **long) == MIS
    f = L.qlinear_paged_attention_shared_workspace_bytes
    assert f(ctypes.byref(c), 1, 8, 1, 1, 1, 1, 1, None) == INV
    assert f(ctypes.byref(c), 1, 8, 1, 1, 1, 0, 1, ctypes.byref(n)) == INV
    assert f(ctypes.byref(c), 1, 8, 1, 1, 1, 1, -1, ctypes.byref(n)) == INV
    assert f(ctypes.byref(c), 0, 8, 0, 0, 0, 1, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert f(ctypes.byref(c), 3, 8, 2, 3, 100, 1, 64, ctypes.byref(n)) == 0 and n.value > 0
    assert _shared(ws=None) == WSP and _shared(ws_bytes=100) == WSP and _shared(ws=FAKE + 8) == MIS


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    exe = str(tmp_path_factory.mktemp("probe") / "view_workspace_probe")
    cmd = [hipcc, "-std=c++20", "-O1", "-x", "hip", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "dequant_matmul_gptq_amd", "csrc"),
           os.path.join(ROOT, "tests", "host", "view_workspace_probe.cpp"), "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([exe], input=text, check=True, capture_output=True, text=True).stdout
        got = [tuple(map(int, line.split())) for line in out.splitlines()]
        assert len(got) == len(cases)
        return got

    return ask


def _call(cache, q_heads, tokens, batch, max_q, max_kv, window=0, sinks=0, groups=0, max_shared=0):
    """Sizes as the entry points hand them on (max_q_len within 1 .. tokens)."""
    return (*cache, tokens, q_heads, batch, max(1, min(max_q, tokens)), max_kv, window, sinks, groups, max_shared)


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("shared", (False, True))
def test_an_answer_covers_smaller_calls(probe, seed, shared):
    rng = random.Random(seed)
    log = lambda hi: int(hi ** rng.random() + 0.5)      # noqa: E731
    for _ in range(25):
        kv = rng.choice((1, 2, 3, 5, 8, 10, 32, 40, 100, 300))
        group = rng.choice((1, 2, 4, 5, 8, 16, 17, 33, 64, 71))
        cache = (rng.choice((64, 128, 256)), rng.choice((16, 8, 6, 4)), kv)
        fixed = () if shared else (rng.choice((0, 1, 100, 1000, 4096)), rng.choice((1, 4, 33, 1000, TOP)))
        top = [log(20000), log(300), log(9000), log(200000)] + ([log(100), log(100000)] if shared else [])
        sizes = lambda t: t[:4] + (([0, 0] + t[4:]) if shared else list(fixed))      # noqa: E731
        cases = [_call(cache, kv * group, *sizes(top))]
        for _ in range(300):
            small = [rng.choice((log(x), max(1, x - rng.randrange(40)), x)) for x in top]
            cases.append(_call(cache, kv * group, *sizes(small)))
        got = probe(cases)
        for case, (need, _) in zip(cases, got):
            assert need <= got[0][1], (cases[0], case)


def test_groups_of_sequences(probe):
    """Rows, lengths and kinds of groups and sequences, with groups that are empty, numbers that are no rows, and
    sequences of no group."""
    rng = random.Random(0)
    cases, want = [], []
    for _ in range(300):
        n, G = rng.randrange(1, 9), rng.randrange(1, 6)
        lens = [rng.randrange(0, 5) for _ in range(n)]
        q = [sum(lens[:i]) for i in range(n + 1)]
        kv = [rng.randrange(0, 300) for _ in range(n)]
        start = sorted(rng.randrange(0, n + 1) for _ in range(G + 1))
        shared = [rng.choice((0, 5, 48, 100, -3)) for _ in range(G)]
        tokens = q[-1] + rng.randrange(3)
        cases.append(("rows", tokens, n, G, *q, *start, *shared, *kv))
        row = []
        for g in range(G):
            s, e = start[g], start[g + 1]
            rows = q[e] - q[s] if shared[g] > 0 else 0
            row.append((q[s], rows, max(0, shared[g]), 0, min(s, n - 1), 1))
        for s in range(n):
            low = next((max(0, shared[g]) for g in range(G) if start[g] <= s < start[g + 1]), 0)
            row.append((q[s], lens[s], kv[s], low, s, 0))
        want.append(row)
    for case, got, w in zip(cases, probe(cases), want):
        got = [got[i:i + 6] for i in range(0, len(got), 6)]
        for a, b in zip(got, w):
            assert a[1:] == b[1:] and (b[1] == 0 or a[0] == b[0]), (case, a, b)
    # numbers that no group, row or length has stay inside the buffers
    bad = (-2 ** 31, -5, 0, 3, 7, 8, 100, TOP)
    cases = [("rows", 8, 3, 2, *(rng.choice(bad) for _ in range(4)), *(rng.choice(bad) for _ in range(3)),
              *(rng.choice(bad) for _ in range(2)), *(rng.choice(bad) for _ in range(3))) for _ in range(2000)]
    for case, got in zip(cases, probe(cases)):
        for q0, n, length, low, row, _ in (got[i:i + 6] for i in range(0, len(got), 6)):
            assert q0 >= 0 and n >= 0 and (n == 0 or q0 + n <= 8), case
            assert 0 <= length <= 16000 and 0 <= low <= 16000 and 0 <= row < 3, case


def test_binding_refuses():
    x = torch.zeros((4, 2, 64), dtype=torch.float16)
    pool = torch.zeros((1, 2, 16, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        dq.paged_attention_shared(dq.KVCache(pool, pool), x, None, None, None)


def test_pool_counts_shared_tokens():
    pool = dq.PagePool(20, 4)
    pool.add("a")
    pool.extend("a", 11)
    assert pool.shared_tokens(["a"]) == 11 and pool.shared_tokens([]) == 0
    pool.fork("a", "b")
    assert pool.shared_tokens(["a", "b"]) == 8      # the last page is a copy
    pool.extend("b", 9)
    pool.fork("b", "c", 16)
    assert pool.shared_tokens("bc") == 16 and pool.shared_tokens("abc") == 8 and pool.shared_tokens("ca") == 8
    pool.add("d")
    assert pool.shared_tokens("abd") == 0
    pool.extend("d", 5)
    assert pool.shared_tokens("da") == 0
    pool.fork("c", "e", 4)
    pool.extend("e", 1)
    assert pool.shared_tokens("ce") == 4
    pool.truncate("c", 12)
    assert pool.shared_tokens("bc") == 12
