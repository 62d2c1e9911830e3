"""Norms of query and key heads with the rotary step, alone and with the append
to a paged cache, against the float64 oracle.

Bound: the sum of D <= 512 squares takes 8 additions in a lane and 6 across
lanes at most, each a relative 2^-24, halved by the square root; with the root,
the division and the two products the normed value is within a relative 2^-20.
The rotation's products and sum add 2^-22 of |a^| + |b^|, the rounding half a
step: |err| <= 2^-11 |y| + (2^-20 + 2^-22) (|a^| + |b^|) + 2^-25.
"""

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
import oracle
from gpu_util import Guarded, device, say

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _x(rng, *shape):
    return rng.standard_normal(shape).astype(np.float16)


def _weight(rng, kind, H, D):
    return (1 + 0.3 * rng.standard_normal((H, D) if kind == "heads" else D)).astype(np.float16)


def _gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device())


def _check(y, x, w, positions, table, rot, interleaved, eps=EPS, what=""):
    n = oracle.decoder.head_norm(x, w, eps)
    ref = oracle.decoder.rope(n, positions, table, rot, interleaved) if rot else n
    i = np.arange(n.shape[-1])
    if interleaved:
        partner = np.where(i < rot, i ^ 1, i)
    else:
        partner = np.where(i < rot // 2, i + rot // 2, np.where(i < rot, i - rot // 2, i))
    amp = np.abs(n) + np.abs(n[..., partner])
    err = np.abs(y.astype(np.float64) - ref)
    bound = 2.0 ** -11 * np.abs(ref) + (2.0 ** -20 + 2.0 ** -22) * amp + 2.0 ** -25
    assert (err <= bound).all(), f"{what}: {(err / bound).max():.3f} bounds"


@pytest.mark.parametrize("D,rot", [(16, 16), (48, 32), (64, 64), (80, 32), (128, 128), (128, 64), (256, 96), (512, 512),
                                   (128, 0), (112, 0)])
@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("T,H,kind", [(1, 1, "one"), (3, 5, "heads"), (40, 32, "one"), (300, 7, "heads")])
def test_norm_rope(D, rot, interleaved, T, H, kind):
    say(f"norm_rope D={D} rot={rot} interleaved={interleaved} T={T} H={H} {kind}")
    rng = np.random.default_rng(D + rot + T)
    x, w = _x(rng, T, H, D), _weight(rng, kind, H, D)
    pos = rng.integers(0, 5000, T).astype(np.int32)
    table = dq.rope_table(5000, rot) if rot else None
    layout = dq.ROPE_INTERLEAVED if interleaved else dq.ROPE_HALF
    xg, wg, pg = _gpu(x), _gpu(w), _gpu(pos)
    tg = table.to(device()) if rot else None
    y = dq.rope(xg, pg if rot else None, tg, layout, norm=wg, eps=EPS)
    _check(y.cpu().numpy(), x, w, pos, table.numpy() if rot else None, rot, interleaved)
    # strided in, strided out, guards around
    fused = torch.full((T, H + 2, D), 5.0, dtype=torch.float16, device=device())
    fused[:, 1:H + 1] = xg
    g = Guarded(T * (H + 1) * D * 2, device())
    out = g.view(torch.float16, (T, H + 1, D))
    before = out[:, H].clone()
    dq.rope(fused[:, 1:H + 1], pg, tg, layout, out=out[:, :H], norm=wg, eps=EPS)
    assert g.intact() and torch.equal(out[:, :H], y)
    assert torch.equal(out[:, H].view(torch.int16), before.view(torch.int16))
    dq.rope(xg, pg, tg, layout, out=xg, norm=wg, eps=EPS)
    assert torch.equal(xg, y)


def test_norm_edges():
    """Rows of zeros, of the smallest and the largest numbers, of NaN; positions outside the table."""
    say("norm edges")
    x = np.zeros((6, 1, 64), np.float16)
    x[1] = 2.0 ** -24
    x[2] = 65504
    x[3, 0, 5] = np.nan
    x[4] = 1
    x[5, 0, 0] = np.inf
    w = np.full(64, 2, np.float16)
    table = dq.rope_table(4, 32)
    pos = np.array([0, 0, 0, 0, 9, 0], np.int32)
    y = dq.rope(_gpu(x), _gpu(pos), table.to(device()), norm=_gpu(w), eps=1e-6).cpu().numpy()
    _check(y[:3], x[:3], w, pos[:3], table.numpy(), 32, False, eps=1e-6)
    assert not y[0].any() and np.abs(y[2] - 2).max() <= 2.0 ** -10
    assert np.isnan(y[3]).all()
    assert np.isnan(y[4, 0, :32]).all() and np.abs(y[4, 0, 32:] - 2).max() <= 2.0 ** -10
    assert np.isnan(y[5, 0, 0]) and not np.nan_to_num(y[5, 0, 32:]).any()


@pytest.mark.parametrize("bits,group", [(16, 32), (8, 32), (8, 128), (6, 64), (4, 32), (4, 128)])
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (128, 128, False), (128, 32, True), (256, 0, False)])
@pytest.mark.parametrize("T,Hq,Hk,kind", [(1, 4, 4, "one"), (17, 5, 1, "heads"), (260, 8, 2, "one"), (300, 24, 8, "heads")])
def test_norm_rope_append(bits, group, D, rot, interleaved, T, Hq, Hk, kind):
    if D % group:
        group = 32
    say(f"norm_rope_append bits={bits} group={group} D={D} rot={rot} T={T} {kind}")
    rng = np.random.default_rng(bits + group + D + T)
    q, k, v = _x(rng, T, Hq, D), _x(rng, T, Hk, D) * 3, _x(rng, T, Hk, D)
    qw, kw = _weight(rng, kind, Hq, D), _weight(rng, kind, Hk, D)
    P, pages = 32, -(-T // 32) + 2
    pos = rng.integers(0, 900, T).astype(np.int32)
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    if T > 1:
        slots[0], slots[T // 2] = -1, pages * P     # padding tokens
    table = dq.rope_table(900, rot) if rot else None
    tg, layout = table.to(device()) if rot else None, dq.ROPE_INTERLEAVED if interleaved else dq.ROPE_HALF
    pg = _gpu(pos) if rot else None
    fused = _gpu(np.concatenate([q, k, v], axis=1))
    qs, ks, vs = fused[:, :Hq], fused[:, Hq:Hq + Hk], fused[:, Hq + Hk:]
    qwg, kwg = _gpu(qw), _gpu(kw)
    kn = dq.rope(ks, pg, tg, layout, norm=kwg, eps=EPS)
    _check(kn.cpu().numpy(), k, kw, pos, table.numpy() if rot else None, rot, interleaved)
    live = [t for t in range(T) if 0 <= slots[t] < pages * P]
    pg_, off = slots[live] // P, slots[live] % P

    def cache():
        c = dq.KVCache.empty(pages, Hk, D, page_size=P, bits=bits, group=group)
        for t in (c.k, c.v, c.k_scales, c.v_scales):
            if t is not None:
                t.fill_(3)
        return c

    def same(c, k_rows, v_rows):
        for pool, scales, x in ((c.k, c.k_scales, k_rows), (c.v, c.v_scales, v_rows)):
            want = np.full(tuple(pool.shape), 3, pool.cpu().numpy().dtype)
            if bits == 16:
                want[pg_, :, off] = x[live]
            else:
                wd, s = oracle.kv_quantize(x[live].reshape(-1, D), bits, group)
                want[pg_, :, off] = wd.view(np.int32).reshape(len(live), Hk, -1)
                ws = np.full(tuple(scales.shape), 3, np.float16)
                ws[pg_, :, off] = s.reshape(len(live), Hk, -1)
                assert np.array_equal(scales.cpu().numpy().view(np.uint16), ws.view(np.uint16))
            kind = np.uint16 if bits == 16 else np.uint32
            assert np.array_equal(pool.cpu().numpy().view(kind), want.view(kind))

    c = cache()
    y = dq.rope_append(c, qs, ks, vs, pg, _gpu(slots), tg, layout, q_norm=qwg, k_norm=kwg, eps=EPS)
    _check(y.cpu().numpy(), q, qw, pos, table.numpy() if rot else None, rot, interleaved)
    same(c, kn.cpu().numpy(), v)
    # the norm of one of the two, and of keys without queries
    c = cache()
    y2 = dq.rope_append(c, qs, ks, vs, pg, _gpu(slots), tg, layout, q_norm=qwg, eps=EPS)
    assert torch.equal(y2, y)
    same(c, (dq.rope(ks, pg, tg, layout) if rot else ks).cpu().numpy(), v)
    c = cache()
    assert dq.rope_append(c, None, ks, vs, pg, _gpu(slots), tg, layout, k_norm=kwg, eps=EPS) is None
    same(c, kn.cpu().numpy(), v)
    c = cache()
    y3 = dq.rope_append(c, qs, ks, vs, pg, _gpu(slots), tg, layout, k_norm=kwg, eps=EPS)
    assert torch.equal(y3, dq.rope(qs, pg, tg, layout) if rot else qs)
    same(c, kn.cpu().numpy(), v)
    # q in place
    dq.rope_append(c, qs, ks, vs, pg, _gpu(slots), tg, layout, q_out=qs, q_norm=qwg, k_norm=kwg, eps=EPS)
    assert torch.equal(qs, y)


def test_norm_rope_append_in_a_graph():
    say("norm_rope_append graph")
    rng = np.random.default_rng(5)
    T, Hq, Hk, D = 5, 8, 2, 128
    q, k, v = (_gpu(_x(rng, T, h, D)) for h in (Hq, Hk, Hk))
    qw, kw = _gpu(_weight(rng, "one", Hq, D)), _gpu(_weight(rng, "one", Hk, D))
    pos, slots, table = _gpu(np.arange(T, dtype=np.int32)), _gpu(np.arange(T, dtype=np.int32)), dq.rope_table(64, D).to(device())
    c, out = dq.KVCache.empty(2, Hk, D, page_size=16), torch.empty_like(q)

    def call():
        return dq.rope_append(c, q, k, v, pos, slots, table, q_out=out, q_norm=qw, k_norm=kw)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        q.copy_(_gpu(_x(rng, T, Hq, D)))
        k.copy_(_gpu(_x(rng, T, Hk, D)))
        pos.add_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), c.k[0, :, :T].clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], c.k[0, :, :T])


def test_norm_rope_on_another_stream():
    say("norm_rope stream")
    rng = np.random.default_rng(6)
    x, w = _gpu(_x(rng, 64, 8, 128)), _gpu(_weight(rng, "one", 8, 128))
    want = dq.rope(x, None, None, norm=w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = dq.rope(x, None, None, norm=w)
    s.synchronize()
    assert torch.equal(y, want)
