"""Host-side tests of the decoder operators: refusals of the C entry points
(made before any launch), the rotary table, the page pool, and pins of the
oracle's functions. No GPU needed."""

import ctypes
import math
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
from dequant_matmul_gptq_amd import _lib
from oracle import decoder_oracle as od

FAKE = 0x10000      # never dereferenced: every call here is refused first
INV, UNS, MIS, WSP = (_lib.ERR_INVALID_ARGUMENT, _lib.ERR_UNSUPPORTED, _lib.ERR_MISALIGNED, _lib.ERR_WORKSPACE)


def _cache(**kw):
    f = dict(k=FAKE, v=FAKE, k_scales=FAKE, v_scales=FAKE, num_pages=4, page_size=32, kv_heads=2, head_dim=128,
             bits=16, group=32)
    f.update(kw)
    return _lib.qlinear_kv_cache(*[f[n] for n, _ in _lib.qlinear_kv_cache._fields_])


def test_struct_size_matches_header():
    assert ctypes.sizeof(_lib.qlinear_kv_cache) == 4 * 8 + 6 * 4


BAD_CACHES = [(dict(k=None), INV), (dict(v=None), INV), (dict(num_pages=0), INV), (dict(kv_heads=0), INV),
              (dict(page_size=48), UNS), (dict(page_size=512), UNS), (dict(head_dim=96), UNS), (dict(bits=5), UNS),
              (dict(bits=8, group=16), UNS), (dict(bits=8, group=128, head_dim=64), UNS),
              (dict(bits=4, k_scales=None), INV), (dict(bits=4, v_scales=FAKE + 2), MIS), (dict(k=FAKE + 8), MIS),
              (dict(num_pages=1 << 30), UNS), (dict(kv_heads=65536), UNS)]

ATT = dict(q=FAKE, q_stride=1024, tokens=3, q_heads=8, batch=1, q_start=FAKE, kv_len=FAKE, block_table=FAKE,
           table_width=4, max_q_len=3, max_kv_len=100, scale=0.1, window=0, out=FAKE, ws=FAKE, ws_bytes=1 << 30)


def _attention(cache=None, **kw):
    a = dict(ATT)
    a.update(kw)
    c = _cache() if cache is None else cache
    return dq.lib().qlinear_paged_attention(ctypes.byref(c), *a.values(), None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_calls_refuse_bad_caches(change, status):
    c = _cache(**change)
    L = dq.lib()
    assert _attention(cache=c) == status
    n = ctypes.c_size_t(0)
    assert L.qlinear_paged_attention_workspace_bytes(ctypes.byref(c), 1, 8, 1, 1, 1, 0, ctypes.byref(n)) == status
    assert L.qlinear_copy_pages(ctypes.byref(c), 1, FAKE, 1, None) == status
    assert L.qlinear_rope_append(ctypes.byref(c), FAKE, 1024, 8, FAKE, 256, FAKE, 256, FAKE, 1024, 1, FAKE, FAKE, FAKE,
                                 8, 64, 0, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INV), (dict(kv_len=None), INV), (dict(block_table=None), INV), (dict(out=None), INV),
    (dict(tokens=-1), INV), (dict(q_heads=0), INV), (dict(batch=-1), INV), (dict(table_width=0), INV),
    (dict(max_q_len=-1), INV), (dict(max_kv_len=-1), INV), (dict(window=-1), INV), (dict(scale=math.inf), INV),
    (dict(scale=math.nan), INV), (dict(q_start=None, batch=2), INV), (dict(q_stride=1016), INV),
    (dict(q_stride=1028), UNS), (dict(q_heads=7, q_stride=2048), UNS), (dict(batch=65536), UNS),
    (dict(tokens=1 << 30), UNS), (dict(q=FAKE + 2), MIS), (dict(out=FAKE + 4), MIS), (dict(kv_len=FAKE + 1), MIS),
    (dict(q_start=FAKE + 2), MIS), (dict(block_table=FAKE + 2), MIS)])
def test_attention_refuses(change, status):
    assert _attention(**change) == status


def test_attention_no_work_and_workspace_query():
    L = dq.lib()
    assert _attention(tokens=0, q=None, out=None) == 0
    assert _attention(batch=0, q=None, out=None) == 0
    assert L.qlinear_paged_attention(None, *ATT.values(), None) == INV
    n = ctypes.c_size_t(77)
    c = _cache()
    f = L.qlinear_paged_attention_workspace_bytes
    assert f(ctypes.byref(c), 0, 8, 0, 0, 0, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert f(ctypes.byref(c), 1, 8, 1, 1, 1, 0, None) == INV
    assert f(ctypes.byref(c), 1, 7, 1, 1, 1, 0, ctypes.byref(n)) == UNS
    # one token over a long cache is split: it needs a workspace, and says so
    assert f(ctypes.byref(c), 1, 8, 1, 1, 100000, 0, ctypes.byref(n)) == 0
    if n.value:
        kw = dict(tokens=1, max_q_len=1, max_kv_len=100000, table_width=4000)
        assert _attention(ws=None, **kw) == WSP
        assert _attention(ws_bytes=n.value - 1, **kw) == WSP
        assert _attention(ws=FAKE + 8, **kw) == MIS


ROPE = dict(x=FAKE, x_stride=256, tokens=2, heads=2, head_dim=128, positions=FAKE, table=FAKE, table_rows=9,
            rot_dim=64, layout=0, out=FAKE, out_stride=256)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INV), (dict(out=None), INV), (dict(positions=None), INV), (dict(table=None), INV),
    (dict(tokens=-1), INV), (dict(heads=-1), INV), (dict(head_dim=0), INV), (dict(rot_dim=0), INV),
    (dict(table_rows=0), INV), (dict(x_stride=248), INV), (dict(out_stride=0), INV), (dict(x_stride=260), UNS),
    (dict(head_dim=120), UNS), (dict(rot_dim=24), UNS), (dict(rot_dim=144), UNS), (dict(layout=2), UNS),
    (dict(head_dim=528, x_stride=2048, out_stride=2048), UNS), (dict(heads=65536), UNS), (dict(tokens=1 << 22), UNS),
    (dict(x=FAKE + 8), MIS), (dict(out=FAKE + 2), MIS), (dict(table=FAKE + 8), MIS), (dict(positions=FAKE + 2), MIS)])
def test_rope_refuses(change, status):
    a = dict(ROPE)
    a.update(change)
    assert dq.lib().qlinear_rope(*a.values(), None) == status


def test_rope_no_work():
    for change in (dict(tokens=0), dict(heads=0)):
        a = dict(ROPE, x=None, out=None)
        a.update(change)
        assert dq.lib().qlinear_rope(*a.values(), None) == 0


APP = dict(q=FAKE, q_stride=1024, q_heads=8, k=FAKE, k_stride=256, v=FAKE, v_stride=256, q_out=FAKE,
           q_out_stride=1024, tokens=2, positions=FAKE, slots=FAKE, table=FAKE, table_rows=9, rot_dim=64, layout=0)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(q_out=None), INV), (dict(slots=None), INV),
    (dict(positions=None), INV), (dict(table=None), INV), (dict(tokens=-1), INV), (dict(q_heads=-1), INV),
    (dict(rot_dim=-16), INV), (dict(k_stride=128), INV), (dict(v_stride=260), UNS), (dict(rot_dim=8), UNS),
    (dict(layout=-1), UNS), (dict(q_heads=65536), UNS), (dict(k=FAKE + 2), MIS), (dict(slots=FAKE + 1), MIS)])
def test_rope_append_refuses(change, status):
    a = dict(APP)
    a.update(change)
    c = _cache()
    assert dq.lib().qlinear_rope_append(ctypes.byref(c), *a.values(), None) == status


def test_copy_pages_refuses():
    L = dq.lib()
    c = _cache()
    for count, pairs, moves, status in ((-1, FAKE, 1, INV), (1, FAKE, -1, INV), (1, None, 1, INV), (1, FAKE + 4, 1, MIS),
                                        (0, None, 5, 0), (1, None, 0, 0)):
        assert L.qlinear_copy_pages(ctypes.byref(c), count, pairs, moves, None) == status
    assert L.qlinear_copy_pages(None, 1, FAKE, 1, None) == INV
    two = (_lib.qlinear_kv_cache * 2)(_cache(), _cache(num_pages=5))
    assert L.qlinear_copy_pages(two, 2, FAKE, 1, None) == UNS


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INV), (dict(weight=None), INV), (dict(y=None), INV), (dict(M=-1), INV), (dict(K=0), INV),
    (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(eps=math.inf), INV), (dict(y=FAKE, ro=FAKE), INV),
    (dict(K=(1 << 24) + 1), UNS), (dict(M=1 << 22), UNS), (dict(x=FAKE + 2), MIS), (dict(r=FAKE + 8), MIS),
    (dict(ro=FAKE + 24), MIS), (dict(M=0, x=None), 0)])
def test_rms_norm_refuses(change, status):
    a = dict(x=FAKE, r=None, weight=FAKE, M=2, K=64, eps=1e-5, y=FAKE + 4096, ro=None)
    a.update(change)
    assert dq.lib().qlinear_rms_norm(*a.values(), None) == status


# ---------------------------------------------------------------- rotary table

def test_rope_table_plain_and_linear():
    t = dq.rope_table(300, 64, base=500.0).numpy().astype(np.float64)
    ang = np.arange(300)[:, None] * od.rope_frequencies(64, 500.0)
    assert t.shape == (300, 32, 2)
    assert np.abs(t[..., 0] - np.cos(ang)).max() < 2 ** -24 and np.abs(t[..., 1] - np.sin(ang)).max() < 2 ** -24
    lin = dq.rope_table(300, 64, base=500.0, scaling=dict(type="linear", factor=4.0)).numpy()
    assert np.abs(lin[::4] - t[:75]).max() < 1e-6       # position 4 p under factor 4 is position p


def test_rope_table_keeps_precision_at_long_positions():
    t = dq.rope_table(1 << 18, 16).numpy()
    p = (1 << 18) - 1
    want = [math.cos(p * 10000.0 ** (-2 * i / 16)) for i in range(8)]
    assert np.abs(t[p, :, 0] - np.array(want)).max() < 1e-6


def _freq(scaling, rot=128, base=10000.0):
    """Frequencies read back from the table's first step (angles below pi)."""
    t = dq.rope_table(2, rot, base=base, scaling=scaling).numpy().astype(np.float64)
    return np.arctan2(t[1, :, 1], t[1, :, 0]), np.hypot(t[1, :, 1], t[1, :, 0])


def test_rope_table_scalings():
    f = od.rope_frequencies(128, 10000.0)
    g, amp = _freq(dict(type="ntk", factor=8.0))
    assert abs(g[0] - 1) < 1e-6 and abs(g[-1] / (f[-1] / 8) - 1) < 1e-4 and np.all(g <= f * (1 + 1e-5))
    # bands: turns over 8192 tokens decide
    g, amp = _freq(dict(type="bands", factor=8.0, original=8192, low=1.0, high=4.0))
    turns = 8192 * f / (2 * np.pi)
    assert np.abs(g / f - 1)[turns > 4].max() < 1e-4 and np.abs(g / f * 8 - 1)[turns < 1].max() < 1e-4
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all((g[mid] < f[mid]) & (g[mid] > f[mid] / 8)) and np.abs(amp - 1).max() < 1e-6
    # yarn: high frequencies kept, low ones divided, cos and sin amplified
    g, amp = _freq(dict(type="yarn", factor=16.0, original=4096))
    turns = 4096 * f / (2 * np.pi)
    assert np.abs(g / f - 1)[turns > 40].max() < 1e-4 and np.abs(g / f * 16 - 1)[turns < 0.8].max() < 1e-4
    assert np.abs(amp - (0.1 * math.log(16) + 1)).max() < 1e-5
    _, amp = _freq(dict(type="yarn", factor=16.0, original=4096, attention=1.0))
    assert np.abs(amp - 1).max() < 1e-6


@pytest.mark.parametrize("args,kw", [((0, 64), {}), ((4, 63), {}), ((4, 0), {}), ((4, 64), dict(base=0.0)),
                                     ((4, 64), dict(scaling=dict(type="cubic"))),
                                     ((4, 64), dict(scaling=dict(type="linear"))),
                                     ((4, 64), dict(scaling=dict(type="linear", factor=0.5))),
                                     ((4, 64), dict(scaling=dict(type="linear", factor=2.0, low=1))),
                                     ((4, 2), dict(scaling=dict(type="ntk", factor=2.0))),
                                     ((4, 64), dict(scaling=dict(type="bands", factor=2.0, original=8, low=4, high=1)))])
def test_rope_table_refuses(args, kw):
    with pytest.raises(ValueError):
        dq.rope_table(*args, **kw)


# ---------------------------------------------------------------- page pool

def _model_check(pool, mem, seqs):
    """Page contents (a dict page -> list of tokens) hold every sequence."""
    P = pool.page_size
    for s, tokens in seqs.items():
        assert pool.length(s) == len(tokens) and len(pool.pages(s)) == -(-len(tokens) // P)
        got = [mem[p][i] for p in pool.pages(s) for i in range(P)][:len(tokens)]
        assert got == tokens, s
    held = {p for s in seqs for p in pool.pages(s)}
    assert pool.free_pages == pool.num_pages - len(held)


@pytest.mark.parametrize("seed", range(6))
def test_page_pool_against_a_model(seed):
    """Random extensions, forks, truncations, frees and compactions, with the
    copies run on a model of the pages' contents."""
    rng = np.random.default_rng(seed)
    P, N = int(rng.integers(1, 5)), 24
    pool = dq.PagePool(N, P)
    mem = [[None] * P for _ in range(N)]
    seqs, names, token = {}, 0, 0

    def run(copies):
        touched = [p for c in copies for p in c]
        assert len(touched) == len(set(touched))
        for s, d in copies:
            mem[d] = list(mem[s])

    for _ in range(400):
        op = rng.choice(["add", "extend", "extend", "fork", "truncate", "free", "compact"])
        s = list(seqs)[int(rng.integers(len(seqs)))] if seqs else None
        if op == "add" and len(seqs) < 6:
            pool.add(names)
            seqs[names] = []
            names += 1
        elif op == "extend" and s is not None:
            n = int(rng.integers(0, 3 * P))
            try:
                slots = pool.extend(s, n)
            except MemoryError:
                _model_check(pool, mem, seqs)
                continue
            assert len(slots) == n
            for x in slots:
                mem[x // P][x % P] = token
                seqs[s].append(token)
                token += 1
        elif op == "fork" and s is not None and len(seqs) < 8:
            try:
                run(pool.fork(s, names))
            except MemoryError:
                continue
            seqs[names] = list(seqs[s])
            names += 1
        elif op == "truncate" and s is not None:
            n = int(rng.integers(0, len(seqs[s]) + 1))
            try:
                pool.truncate(s, n)
            except ValueError:
                continue
            del seqs[s][n:]
        elif op == "free" and s is not None:
            pool.free(s)
            del seqs[s]
        elif op == "compact":
            run(pool.compact())
            held = {p for x in seqs for p in pool.pages(x)}
            assert held == set(range(len(held)))
        _model_check(pool, mem, seqs)


def test_page_pool_refuses():
    with pytest.raises(ValueError):
        dq.PagePool(0, 16)
    p = dq.PagePool(2, 4)
    p.add("a")
    with pytest.raises(ValueError):
        p.add("a")
    with pytest.raises(MemoryError):
        p.extend("a", 9)
    assert p.length("a") == 0 and p.free_pages == 2
    assert p.extend("a", 5) == [0, 1, 2, 3, 4]
    with pytest.raises(MemoryError):
        p.fork("a", "b")
    with pytest.raises(ValueError):
        p.extend("a", -1)
    with pytest.raises(ValueError):
        p.truncate("a", 6)
    with pytest.raises(KeyError):
        p.extend("zz", 1)
    p.truncate("a", 4)
    assert p.fork("a", "b") == [] and p.pages("b") == [0]
    with pytest.raises(ValueError):
        p.truncate("b", 3)
    p.free("a")
    assert p.free_pages == 1
    p.truncate("b", 3)


# ---------------------------------------------------------------- oracle pins

def test_oracle_attention_pins():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((6, 1, 4))
    # equal keys: the mean of the values seen
    o, w, total = od.attention(np.ones((2, 2, 4)), np.ones((6, 1, 4)), v, 0.3)
    assert np.allclose(o[0, 1], v[:5, 0].mean(0)) and np.allclose(o[1, 0], v[:, 0].mean(0))
    assert np.allclose(w[1, 0], np.abs(v[:, 0]).mean(0)) and np.allclose(total, [[5, 5], [6, 6]])
    o, _, _ = od.attention(np.ones((1, 1, 4)), np.ones((6, 1, 4)), v, 0.3, window=2)
    assert np.allclose(o[0, 0], v[4:, 0].mean(0))
    # two tokens: the logistic function of the score difference
    k = np.array([[[1.0, 0.0]], [[0.0, 2.0]]])
    q = np.array([[[0.5, 1.5]]])
    o, _, _ = od.attention(q, k, np.array([[[1.0, 0.0]], [[0.0, 1.0]]]), 2.0)
    p = 1 / (1 + math.exp(2.0 * (3.0 - 0.5)))
    assert np.allclose(o[0, 0], [p, 1 - p])
    # heads: query head h reads h // 2
    k = rng.standard_normal((3, 2, 4))
    q = rng.standard_normal((1, 4, 4))
    o, _, _ = od.attention(q, k, k, 1.0)
    o1, _, _ = od.attention(q[:, 2:], k[:, 1:], k[:, 1:], 1.0)
    assert np.allclose(o[:, 2:], o1)
    o, _, _ = od.attention(rng.standard_normal((3, 1, 4)), k[:1, :1], k[:1, :1], 1.0)
    assert not o[:2].any() and np.allclose(o[2, 0], k[0, 0])


def test_oracle_rope_pins():
    t = np.zeros((2, 2, 2))
    t[0, :, 0] = 1.0                    # angle 0
    t[1, 0], t[1, 1] = (0.0, 1.0), (-1.0, 0.0)      # 90 and 180 degrees
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    assert np.array_equal(od.rope(x, [0], t, 4, False), x)
    assert np.array_equal(od.rope(x, [1], t, 4, False), [[[-3.0, -2.0, 1.0, -4.0, 9.0]]])
    assert np.array_equal(od.rope(x, [1], t, 4, True), [[[-2.0, 1.0, -3.0, -4.0, 9.0]]])


def test_oracle_rms_norm_pins():
    y, h = od.rms_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    r = math.sqrt(12.5)
    assert np.allclose(y, [[3 / r, 8 / r]]) and h.dtype == np.float16
    y, h = od.rms_norm(np.array([[2.0, 5.0]]), np.array([1.0, 2.0]), 0.0, np.array([[1.0, -1.0]]))
    assert np.allclose(y, [[3 / r, 8 / r]]) and h.tolist() == [[3.0, 4.0]]


@pytest.mark.parametrize("cache,change", [
    (dict(kv_heads=4097), dict(q_heads=4097, q_stride=4097 * 128)),
    ({}, dict(tokens=(1 << 26) + 1)),                                  # tokens * q_heads past 2^29
    (dict(kv_heads=128), dict(q_heads=128, q_stride=128 * 128, batch=32769)),   # batch * kv_heads past 2^22
    ({}, dict(batch=8193, table_width=32768))])                        # slots of all tables past 2^33
def test_attention_refuses_what_its_indexes_cannot_hold(cache, change):
    assert _attention(cache=_cache(**cache), **change) == UNS


@pytest.mark.parametrize("change", [dict(M=1 << 22), dict(K=(1 << 24) + 8)])
def test_rms_norm_refuses_what_its_indexes_cannot_hold(change):
    a = dict(x=FAKE, residual=None, weight=FAKE, M=1, K=64, eps=1e-5, out=FAKE, residual_out=None)
    a.update(change)
    assert dq.lib().qlinear_rms_norm(*a.values(), None) == UNS


def test_binding_refuses_host_tensors():
    """Calls whose operands are all in host memory, so that their devices agree."""
    x, w = torch.zeros((4, 2, 64), dtype=torch.float16), torch.ones(64, dtype=torch.float16)
    pos, table = torch.zeros(4, dtype=torch.int32), dq.rope_table(8, 64)
    for call in (lambda: dq.rms_norm(x, w), lambda: dq.rms_norm(x, w, residual=x, out=x, residual_out=x.clone()),
                 lambda: dq.rope(x, pos, table), lambda: dq.rope(x[:0], pos[:0], table),
                 lambda: dq.rope(x.to("meta"), pos, table), lambda: dq.KVCache(x[None], x[None])):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_binding_passes_no_number_cut_to_32_bits():
    """Past 32 bits a bound counts as the largest one and a size is refused."""
    cache = SimpleNamespace(ref=ctypes.byref(_cache()))
    need = lambda *sizes: dq.paged_attention_workspace_bytes(cache, *sizes)      # noqa: E731
    top = 2 ** 31 - 1
    assert need(8, 8, 2, 4, 2 ** 32, 0) == need(8, 8, 2, 4, top, 0) > 0
    assert need(8, 8, 2, 2 ** 32 + 1, 5000, 0) == need(8, 8, 2, top, 5000, 0)
    assert need(8, 8, 2, 4, 5000, 2 ** 32 + 64) == need(8, 8, 2, 4, 5000, top) != need(8, 8, 2, 4, 5000, 64)
    for sizes, status in (((2 ** 32 + 8, 8, 2, 4, 5000), UNS), ((8, 2 ** 32 + 8, 2, 4, 5000), UNS),
                          ((8, 8, 2 ** 32 + 2, 4, 5000), UNS), ((8, 8, 2, -2 ** 32, 5000), INV),
                          ((8, 8, 2, 4, 5000, 1 - 2 ** 32), INV)):
        with pytest.raises(dq.QlinearError) as e:
            need(*sizes)
        assert e.value.status == status, sizes


def test_page_pool_rolls_back_inside_a_shared_page():
    """Drafts rejected just after a fork at a page boundary: what the fork shares cannot be cut, but forked up to a length."""
    pool = dq.PagePool(6, 4)
    mem = {}
    pool.add("a")
    for i, s in enumerate(pool.extend("a", 8)):
        mem[s] = i
    assert pool.fork("a", "b") == []
    with pytest.raises(ValueError, match="fork"):
        pool.truncate("b", 6)
    copies = pool.fork("b", "c", 6)
    assert len(copies) == 1 and copies[0][0] == pool.pages("a")[1] and pool.length("c") == 6
    for src, dst in copies:
        mem.update({dst * 4 + i: mem[src * 4 + i] for i in range(4)})
    pool.free("b")
    new = pool.extend("c", 3)
    for i, s in enumerate(new):
        mem[s] = 100 + i
    read = lambda seq: [mem.get(p * 4 + i) for p in pool.pages(seq) for i in range(4)][:pool.length(seq)]    # noqa: E731
    assert read("c") == [0, 1, 2, 3, 4, 5, 100, 101, 102] and read("a") == list(range(8))
    assert pool.pages("c")[0] == pool.pages("a")[0]
    # at a boundary nothing is copied; up to nothing, nothing is held
    assert pool.fork("c", "d", 8) == [] and pool.pages("d") == pool.pages("c")[:2]
    assert pool.fork("c", "e", 0) == [] and pool.pages("e") == [] and pool.length("e") == 0
    assert pool.fork("c", "f", 9) and pool.length("f") == 9
    used = pool.num_pages - pool.free_pages
    assert used == len({p for s in pool.sequences() for p in pool.pages(s)}) == 5
    for length in (10, -1):
        with pytest.raises(ValueError):
            pool.fork("c", "g", length)
    assert "g" not in pool.sequences() and pool.num_pages - pool.free_pages == used
    for s in pool.sequences():
        pool.free(s)
    assert pool.free_pages == 6


@pytest.mark.parametrize("seed", range(4))
def test_page_pool_forks_of_any_length_against_a_model(seed):
    rng = np.random.default_rng(seed)
    P, N, token, names = int(rng.integers(1, 6)), 30, 0, 1
    pool, mem, seqs = dq.PagePool(N, P), [[None] * P for _ in range(N)], {0: []}
    pool.add(0)
    for _ in range(300):
        s = list(seqs)[int(rng.integers(len(seqs)))]
        op = rng.choice(["extend", "fork", "free", "compact"])
        copies = []
        try:
            if op == "extend":
                for x in pool.extend(s, int(rng.integers(0, 2 * P))):
                    mem[x // P][x % P] = token
                    seqs[s].append(token)
                    token += 1
            elif op == "fork" and len(seqs) < 8:
                n = int(rng.integers(0, len(seqs[s]) + 1))
                copies = pool.fork(s, names, n)
                seqs[names] = seqs[s][:n]
                names += 1
            elif op == "free" and len(seqs) > 1:
                pool.free(s)
                del seqs[s]
            elif op == "compact":
                copies = pool.compact()
        except MemoryError:
            pass
        for src, dst in copies:
            mem[dst] = list(mem[src])
        _model_check(pool, mem, seqs)


def test_calls_run_with_their_tensors_gpu_as_the_current_one(monkeypatch):
    """Also where another one is: the default stream's handle is 0 on every GPU. (No GPU: the library and the
    device calls stand-ins.)"""
    from dequant_matmul_gptq_amd import decoder
    state = dict(current=0, calls=[])

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, state["current"] = state["current"], self.device

        def __exit__(self, *_):
            state["current"] = self.before

    class Tensor:
        dtype, shape = torch.float16, torch.Size((3, 64))

        def __init__(self, *shape):
            self.shape = torch.Size(shape)

        def get_device(self):
            return 2

        def is_contiguous(self):
            return True

        def dim(self):
            return len(self.shape)

        def numel(self):
            return self.shape.numel()

        def data_ptr(self):
            return FAKE

    def norm(*args):
        state["calls"].append((state["current"], args[-1]))
        return state.get("status", 0)

    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(decoder, "_current_gpu", lambda: state["current"], raising=False)
    monkeypatch.setattr(decoder, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(decoder, "lib", lambda: SimpleNamespace(qlinear_rms_norm=norm))
    x, w, y = Tensor(3, 64), Tensor(64), Tensor(3, 64)
    assert dq.rms_norm(x, w, out=y) is y
    assert state["calls"] == [(2, 1002)] and state["current"] == 0
    state["status"] = INV
    with pytest.raises(dq.QlinearError):
        dq.rms_norm(x, w, out=y)
    assert state["calls"][1:] == [(2, 1002)] and state["current"] == 0
    state.update(status=0, current=2)
    dq.rms_norm(x, w, out=y)
    assert state["calls"][2:] == [(2, 1002)] and state["current"] == 2
