"""Rotary positions, the append to a paged cache, page copies and the norm
against the float64 oracle.

Bounds: rotation has two products and a sum in float32 and one float16
rounding: |err| <= 2^-11 |y| + 2^-22 (|a| + |b|) + 2^-25. The norm has a
float32 sum of K squares (relative error below 2^-17 for K up to 32768 at the
summation depths used), a square root, a division and two products, then one
rounding: |err| <= (2^-11 + 2^-15) |y| + 2^-25. Cache contents are compared bit
for bit with the codec's oracle, on the values the rotation returned.
"""

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
import oracle
from gpu_util import Guarded, device, say

pytestmark = pytest.mark.gpu


def _x(rng, *shape):
    return rng.standard_normal(shape).astype(np.float16)


def _gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device())


def _check_rotation(y, x, positions, table, rot, interleaved):
    ref = oracle.decoder.rope(x, positions, table, rot, interleaved)
    err = np.abs(y.astype(np.float64) - ref)
    # |a| + |b| of an element's pair, at most the token's largest sum of two
    amp = 2 * np.abs(x.astype(np.float64)).max()
    assert (err <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -22 * amp + 2.0 ** -25).all(), err.max()
    assert np.array_equal(y[..., rot:].view(np.uint16), x[..., rot:].view(np.uint16))


@pytest.mark.parametrize("D,rot", [(16, 16), (64, 64), (64, 16), (80, 32), (128, 128), (128, 64), (256, 96),
                                   (512, 512)])
@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("T,H", [(1, 1), (3, 5), (40, 32), (300, 7)])
def test_rope(D, rot, interleaved, T, H):
    say(f"rope D={D} rot={rot} interleaved={interleaved} T={T} H={H}")
    rng = np.random.default_rng(D + rot + T)
    x = _x(rng, T, H, D)
    pos = rng.integers(0, 5000, T).astype(np.int32)
    table = dq.rope_table(5000, rot)
    layout = dq.ROPE_INTERLEAVED if interleaved else dq.ROPE_HALF
    xg, tg, pg = _gpu(x), table.to(device()), _gpu(pos)
    y = dq.rope(xg, pg, tg, layout)
    _check_rotation(y.cpu().numpy(), x, pos, table.numpy(), rot, interleaved)
    # strided in, strided out, guards around
    fused = torch.full((T, H + 2, D), 5.0, dtype=torch.float16, device=device())
    fused[:, 1:H + 1] = xg
    g = Guarded(T * (H + 1) * D * 2, device())
    out = g.view(torch.float16, (T, H + 1, D))
    before = out[:, H].clone()
    dq.rope(fused[:, 1:H + 1], pg, tg, layout, out=out[:, :H])
    assert g.intact() and torch.equal(out[:, :H], y)
    assert torch.equal(out[:, H].view(torch.int16), before.view(torch.int16))
    # in place
    dq.rope(xg, pg, tg, layout, out=xg)
    assert torch.equal(xg, y)


def test_rope_positions_outside_the_table_give_nan():
    say("rope positions")
    x = torch.ones((3, 2, 64), dtype=torch.float16, device=device())
    y = dq.rope(x, _gpu(np.array([5, -1, 10], np.int32)), dq.rope_table(10, 32).to(device()))
    y = y.cpu().numpy()
    assert np.isfinite(y[0]).all() and np.isnan(y[1:, :, :32]).all() and (y[:, :, 32:] == 1).all()


@pytest.mark.parametrize("bits,group", [(16, 32), (8, 32), (8, 128), (6, 32), (6, 64), (4, 32), (4, 128)])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 64, True), (128, 32, False), (256, 256, True)])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 4, 4), (17, 5, 1), (260, 8, 2)])
def test_rope_append(bits, group, D, rot, interleaved, T, Hq, Hk):
    say(f"rope_append bits={bits} group={group} D={D} rot={rot} interleaved={interleaved} T={T}")
    rng = np.random.default_rng(bits + group + D + T)
    q, k, v = _x(rng, T, Hq, D), _x(rng, T, Hk, D) * 3, _x(rng, T, Hk, D)
    P = 32
    pages = -(-T // P) + 2
    pos = rng.integers(0, 900, T).astype(np.int32)
    slots = rng.permutation(pages * P)[:T].astype(np.int32)
    if T > 1:
        slots[0], slots[T // 2] = -1, pages * P     # padding tokens
    table = dq.rope_table(900, rot)
    c = dq.KVCache.empty(pages, Hk, D, page_size=P, bits=bits, group=group)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        if t is not None:
            t.fill_(3)
    tg, layout = table.to(device()), dq.ROPE_INTERLEAVED if interleaved else dq.ROPE_HALF
    # a fused projection's output: q, k and v side by side
    fused = _gpu(np.concatenate([q, k, v], axis=1))
    qs, ks, vs = fused[:, :Hq], fused[:, Hq:Hq + Hk], fused[:, Hq + Hk:]
    y = dq.rope_append(c, qs, ks, vs, _gpu(pos), _gpu(slots), tg, layout)
    _check_rotation(y.cpu().numpy(), q, pos, table.numpy(), rot, interleaved)
    kr = dq.rope(ks, _gpu(pos), tg, layout).cpu().numpy()
    live = [t for t in range(T) if 0 <= slots[t] < pages * P]
    pg, off = slots[live] // P, slots[live] % P
    for pool, scales, x in ((c.k, c.k_scales, kr), (c.v, c.v_scales, v)):
        want = np.full(tuple(pool.shape), 3, pool.cpu().numpy().dtype)
        if bits == 16:
            want[pg, :, off] = x[live]
        else:
            w, s = oracle.kv_quantize(x[live].reshape(-1, D), bits, group)
            want[pg, :, off] = w.view(np.int32).reshape(len(live), Hk, -1)
            ws = np.full(tuple(scales.shape), 3, np.float16)
            ws[pg, :, off] = s.reshape(len(live), Hk, -1)
            assert np.array_equal(scales.cpu().numpy().view(np.uint16), ws.view(np.uint16))
        got = pool.cpu().numpy()
        assert np.array_equal(got.view(np.uint16 if bits == 16 else np.uint32),
                              want.view(np.uint16 if bits == 16 else np.uint32))
    # q rotated in place, and the append without rotation or q
    dq.rope_append(c, qs, ks, vs, _gpu(pos), _gpu(slots), tg, layout, q_out=qs)
    assert torch.equal(qs, y)
    c2 = dq.KVCache.empty(pages, Hk, D, page_size=P, bits=bits, group=group)
    assert dq.rope_append(c2, None, vs, vs, None, _gpu(slots), None) is None
    i = torch.from_numpy(pg.astype(np.int64)).to(device()), slice(None), torch.from_numpy(off.astype(np.int64)).to(device())
    assert torch.equal(c2.k[i].view(torch.int16), c2.v[i].view(torch.int16))
    assert torch.equal(c2.v[i].view(torch.int16), c.v[i].view(torch.int16))


@pytest.mark.parametrize("bits", (16, 8, 4))
def test_append_propagates_nan(bits):
    """A NaN in a block is not lost in its codes."""
    say(f"append nan bits={bits}")
    x = np.ones((2, 1, 64), np.float16)
    x[1, 0, 40] = np.nan
    c = dq.KVCache.empty(1, 1, 64, page_size=16, bits=bits, group=32)
    dq.rope_append(c, None, _gpu(x), _gpu(x), None, _gpu(np.array([0, 1], np.int32)), None)
    v = c.v if bits == 16 else dq.kv_dequant(c.v, c.v_scales, 64, bits, 32)
    v = v.cpu().numpy()[0, 0]
    assert (v[0] == 1).all() and (v[1, :32] == 1).all() and np.isnan(v[1, 40])


@pytest.mark.parametrize("bits,group", [(16, 32), (8, 128), (6, 32), (4, 64)])
@pytest.mark.parametrize("layers,heads,P", [(1, 1, 16), (3, 5, 32), (70, 2, 16), (2, 32, 256)])
def test_copy_pages(bits, group, layers, heads, P):
    say(f"copy_pages bits={bits} layers={layers} heads={heads} P={P}")
    rng = np.random.default_rng(layers)
    caches = [dq.KVCache.empty(9, heads, 128, page_size=P, bits=bits, group=group) for _ in range(layers)]
    pools = [t for c in caches for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None]
    for t in pools:
        t.view(torch.int16).copy_(torch.randint(-30000, 30000, t.view(torch.int16).shape, dtype=torch.int16))
    want = [t.clone() for t in pools]
    pairs = rng.permutation(9)[:8].reshape(4, 2).astype(np.int32)
    for s, d in pairs[:3]:
        for w in want:
            w[d] = w[s]
    pairs[3] = (9, pairs[3, 1]) if layers % 2 else (pairs[3, 0], -1)     # outside the pool: skipped
    dq.copy_pages(caches, _gpu(pairs))
    for t, w in zip(pools, want):
        assert torch.equal(t.view(torch.int16), w.view(torch.int16))
    dq.copy_pages(caches, _gpu(pairs[:0]))
    dq.copy_pages([], _gpu(pairs))
    for t, w in zip(pools, want):
        assert torch.equal(t.view(torch.int16), w.view(torch.int16))


def test_copy_pages_refuses_mixed_shapes():
    a = dq.KVCache.empty(4, 2, 64, page_size=16)
    for b in (dq.KVCache.empty(5, 2, 64, page_size=16), dq.KVCache.empty(4, 2, 64, page_size=16, bits=8)):
        with pytest.raises(dq.QlinearError) as e:
            dq.copy_pages([a, b], _gpu(np.array([[0, 1]], np.int32)))
        assert e.value.status == dq._lib.ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        dq.copy_pages([a], _gpu(np.array([0, 1], np.int32)))
    with pytest.raises(ValueError):
        dq.copy_pages([a], _gpu(np.array([[0, 1]], np.int64)))


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 8), (2, 511), (9, 512), (4, 520), (1, 2048), (700, 2056), (6, 4096),
                                 (3, 5120), (1, 8192), (5, 8200), (2, 16384), (1, 20000), (2, 32768), (2, 32776),
                                 (1, 100001), (1500, 64), (1030, 4096)])
@pytest.mark.parametrize("residual", (False, True))
def test_rms_norm(M, K, residual):
    say(f"rms_norm M={M} K={K} residual={residual}")
    rng = np.random.default_rng(M + K)
    x = _x(rng, M, K)
    r = (_x(rng, M, K) * np.float16(4)) if residual else None
    w = (1 + 0.2 * rng.standard_normal(K)).astype(np.float16)
    ref, h = oracle.decoder.rms_norm(x, w, 1e-5, r)
    dev = device()
    og, hg = Guarded(M * K * 2, dev), Guarded(M * K * 2, dev)
    out, hout = og.view(torch.float16, (M, K)), hg.view(torch.float16, (M, K))
    xg, rg, wg = _gpu(x), None if r is None else _gpu(r), _gpu(w)
    dq.rms_norm(xg, wg, 1e-5, residual=rg, out=out, residual_out=hout)
    assert og.intact() and hg.intact()
    assert np.array_equal(hout.cpu().numpy().view(np.uint16), h.view(np.uint16))
    y = out.cpu().numpy().astype(np.float64)
    err = np.abs(y - ref)
    assert (err <= (2.0 ** -11 + 2.0 ** -15) * np.abs(ref) + 2.0 ** -25).all(), (err / np.maximum(np.abs(ref), 1e-9)).max()
    # without the sum written out, and with outputs over the inputs
    assert torch.equal(dq.rms_norm(xg, wg, 1e-5, residual=rg), out)
    if residual:
        a, b = xg.clone(), rg.clone()
        dq.rms_norm(a, wg, 1e-5, residual=b, out=a, residual_out=b)
        assert torch.equal(a, out) and torch.equal(b, hout)
        a, b = xg.clone(), rg.clone()
        dq.rms_norm(a, wg, 1e-5, residual=b, out=b, residual_out=a)
        assert torch.equal(b, out) and torch.equal(a, hout)
    a = xg.clone()
    dq.rms_norm(a, wg, 1e-5, residual=rg, out=a)
    assert torch.equal(a, out)


def test_rms_norm_special_values():
    say("rms_norm special")
    x = np.zeros((4, 64), np.float16)
    x[1] = 60000.0
    x[2, 3] = np.inf
    x[3, 5] = np.nan
    w = np.ones(64, np.float16)
    y = dq.rms_norm(_gpu(x), _gpu(w), 1e-5).cpu().numpy()
    assert not y[0].any() and np.abs(y[1] - 1).max() < 1e-3
    assert np.isnan(y[2, 3]) and not y[2, :3].any() and np.isnan(y[3]).all()
    # eps == 0 on a row of zeros is 0 / 0
    assert np.isnan(dq.rms_norm(_gpu(x[:1]), _gpu(w), 0.0).cpu().numpy()).all()
    # a batch of no rows
    assert dq.rms_norm(torch.empty((0, 64), dtype=torch.float16, device=device()), _gpu(w)).shape == (0, 64)


def test_binding_refuses_wrong_tensors():
    dev = device()
    x = torch.zeros((4, 2, 64), dtype=torch.float16, device=dev)
    w = torch.ones(64, dtype=torch.float16, device=dev)
    for bad in (dict(x=x.float()), dict(weight=w[:32]), dict(residual=x[:2]), dict(x=x.cpu()),
                dict(x=x.transpose(0, 1))):
        args = dict(x=x, weight=w)
        args.update(bad)
        with pytest.raises(ValueError):
            dq.rms_norm(**args)
    y = torch.empty_like(x)
    with pytest.raises(dq.QlinearError):
        dq.rms_norm(x, w, residual=x, out=y, residual_out=y)
    with pytest.raises(dq.QlinearError):
        dq.rms_norm(x, w, eps=-1.0)
    pos, table = torch.zeros(4, dtype=torch.int32, device=dev), dq.rope_table(8, 64, device=dev)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:2]), dict(table=table.double()), dict(table=table.cpu()),
                dict(x=x.transpose(0, 1)), dict(out=x[:3])):
        args = dict(x=x, positions=pos, table=table)
        args.update(bad)
        with pytest.raises(ValueError):
            dq.rope(**args)
    with pytest.raises(dq.QlinearError) as e:
        dq.rope(x, pos, dq.rope_table(8, 40, device=dev))       # rot_dim 40 is no multiple of 16
    assert e.value.status == dq._lib.ERR_UNSUPPORTED
    c = dq.KVCache.empty(2, 2, 64, page_size=16)
    with pytest.raises(ValueError):
        dq.rope_append(c, None, x[:, :1], x, pos, pos, table)
    with pytest.raises(ValueError):
        dq.rope_append(c, None, x, x, None, pos, table)


def test_rms_norm_refuses_rows_past_32_bits():
    say("rms_norm rows past 32 bits")
    x = torch.empty((2 ** 32 + 5, 1), dtype=torch.float16, device=device())
    out = torch.empty_like(x)
    with pytest.raises(dq.QlinearError) as e:
        dq.rms_norm(x, torch.ones(1, dtype=torch.float16, device=device()), out=out)
    assert e.value.status == dq._lib.ERR_UNSUPPORTED
