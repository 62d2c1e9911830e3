"""Attention over a paged cache against the float64 oracle.

Error bound per output element, from the arithmetic: the softmax weights are
rounded to float16 (relative 2^-11, or absolute 2^-25 of the largest weight for
tiny ones, of which there are at most L), scores and sums are float32 over at
most 256 products and L terms (together below 2^-13 relative in a weight at
these sizes), and the output is rounded once (2^-11 relative, 2^-25 absolute).
So with w = sum_t p_t |v_t|, S = sum_t exp(s_t - max s):
  |err| <= 2^-11 |o| + (2^-11 + 2^-12) w + 2^-25 (1 + L max|v| / S)
"""

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
import oracle
from gpu_util import Guarded, device, say

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences of random keys and values in a paged cache whose other slots
    hold NaN, with pages in random order."""

    def __init__(self, Hq, Hk, D, P, bits, group, q_lens, kv_lens, seed=0, spread=1.0, width_extra=1):
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.Hq, self.Hk, self.D, self.P, self.bits, self.group = Hq, Hk, D, P, bits, group
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        self.q = [(rng.standard_normal((n, Hq, D)) * spread).astype(np.float16) for n in q_lens]
        self.k = [(rng.standard_normal((L, Hk, D)) * rng.uniform(0.5, 1.5, D)).astype(np.float16) for L in kv_lens]
        self.v = [rng.standard_normal((L, Hk, D)).astype(np.float16) for L in kv_lens]
        need = [-(-L // P) for L in kv_lens]
        self.pages = sum(need) + 2
        order = rng.permutation(self.pages)
        W = max(need + [1]) + width_extra
        self.table = np.full((len(kv_lens), W), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.fill()

    def slots(self, b):
        t = np.arange(self.kv_lens[b])
        return self.table[b, t // self.P], t % self.P

    def fill(self):
        """The pools on the device, and self.kv: the float64 values they hold."""
        dev = device()
        shape = (self.pages, self.Hk, self.P)
        self.kv = []
        pools = {}
        for name, xs in (("k", self.k), ("v", self.v)):
            vals = []
            if self.bits == 16:
                pool = np.full(shape + (self.D,), np.nan, np.float16)
            else:
                pool = np.full(shape + (self.D * self.bits // 32,), -1, np.int32)
                sc = np.full(shape + (self.D // self.group,), np.nan, np.float16)
            for b, x in enumerate(xs):
                pg, off = self.slots(b)
                if self.bits == 16:
                    pool[pg, :, off] = x
                    vals.append(x.astype(np.float64))
                elif len(x):
                    w, s = oracle.kv_quantize(x.reshape(-1, self.D), self.bits, self.group)
                    pool[pg, :, off] = w.view(np.int32).reshape(len(x), self.Hk, -1)
                    sc[pg, :, off] = s.reshape(len(x), self.Hk, -1)
                    vals.append(oracle.kv_dequantize(w, s, self.D, self.bits, self.group).astype(np.float64)
                                .reshape(x.shape))
                else:
                    vals.append(x.astype(np.float64))
            pools[name] = torch.from_numpy(pool).to(dev)
            if self.bits != 16:
                pools[name + "_scales"] = torch.from_numpy(sc).to(dev)
            self.kv.append(vals)
        self.cache = dq.KVCache(pools["k"], pools["v"], pools.get("k_scales"), pools.get("v_scales"),
                                head_dim=self.D)

    def run(self, window=0, scale=None, uniform=False, q=None, out=None, **kw):
        dev = device()
        qt = torch.from_numpy(np.concatenate(self.q)).to(dev) if q is None else q
        starts = None if uniform else torch.tensor(np.concatenate([[0], np.cumsum(self.q_lens)]), dtype=torch.int32,
                                                   device=dev)
        o = dq.paged_attention(self.cache, qt, torch.from_numpy(self.table).to(dev),
                               torch.tensor(self.kv_lens, dtype=torch.int32, device=dev), starts, window=window,
                               scale=scale, out=out, **kw)
        torch.cuda.synchronize()
        return o.float().cpu().numpy().astype(np.float64)

    def check(self, o, window=0, scale=None, what=""):
        scale = self.D ** -0.5 if scale is None else scale
        at = 0
        for b, n in enumerate(self.q_lens):
            ref, w, total = oracle.decoder.attention(self.q[b], self.kv[0][b], self.kv[1][b], scale, window)
            got = o[at:at + n]
            at += n
            vmax = np.abs(self.kv[1][b]).max() if self.kv_lens[b] else 0.0
            tiny = self.kv_lens[b] * vmax / np.maximum(total, 1.0)
            bound = 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -12) * w + 2.0 ** -25 * (1 + tiny[..., None])
            assert np.isfinite(got).all(), f"{what} sequence {b}: non-finite output"
            err = np.abs(got - ref)
            assert (err <= bound).all(), f"{what} sequence {b}: error {err.max():.3e}, {(err / bound).max():.2f} bounds"


HEADS = [(4, 4), (8, 1), (6, 2), (16, 1), (20, 4), (33, 1)]


@pytest.mark.parametrize("bits,group", [(16, 128), (8, 64), (8, 128), (6, 32), (6, 128), (4, 32), (4, 64), (4, 128)])
@pytest.mark.parametrize("P", (16, 256))
def test_single_tokens(bits, group, P):
    """One new token per sequence, lengths around the tile and page edges."""
    say(f"attention decode bits={bits} group={group} P={P}")
    b = Batch(8, 2, 128, P, bits, group, [1] * 9, [1, 2, 15, 16, 17, 31, 33, 257, 700], seed=bits + group + P)
    b.check(b.run())
    b.check(b.run(window=20), window=20)


@pytest.mark.parametrize("Hq,Hk", HEADS)
@pytest.mark.parametrize("D", (64, 128, 256))
def test_head_layouts(Hq, Hk, D):
    say(f"attention heads {Hq}/{Hk} D={D}")
    for bits, group, P in ((16, 64, 32), (4, 64, 64)):
        b = Batch(Hq, Hk, D, P, bits, group, [1, 3, 1], [65, 130, 7], seed=Hq + D)
        b.check(b.run(), what=f"bits={bits}")


@pytest.mark.parametrize("n,past", [(2, 0), (7, 100), (16, 16), (33, 5), (64, 0), (65, 63), (127, 129), (200, 300)])
@pytest.mark.parametrize("bits,group", [(16, 64), (8, 32), (6, 64), (4, 64)])
def test_chunks(n, past, bits, group):
    say(f"attention chunk n={n} past={past} bits={bits}")
    b = Batch(4, 2, 64, 32, bits, group, [n], [n + past], seed=n + past + bits)
    b.check(b.run())
    b.check(b.run(window=50), window=50)
    b.check(b.run(window=1), window=1)


@pytest.mark.parametrize("D,bits", [(128, 16), (128, 4), (256, 16), (256, 6)])
def test_chunks_wide_heads(D, bits):
    say(f"attention chunk D={D} bits={bits}")
    b = Batch(8, 2, D, 64, bits, 64, [150, 37], [300, 37], seed=D + bits)
    b.check(b.run())


@pytest.mark.parametrize("bits", (16, 4))
def test_mixed_batch(bits):
    """Prompts, drafts, single tokens, and sequences without new tokens, in one call."""
    say(f"attention mixed bits={bits}")
    b = Batch(8, 2, 64, 16, bits, 32, [130, 1, 5, 0, 1, 70, 0, 2], [130, 333, 40, 12, 1, 500, 0, 2], seed=bits)
    b.check(b.run())
    b.check(b.run(window=64), window=64)
    b.check(b.run(max_q_len=130, max_kv_len=500))


def test_long_split():
    """Lengths that are split over workgroups, ragged, with small and large tables."""
    say("attention long")
    b = Batch(4, 1, 128, 256, 16, 128, [1, 1, 1, 4], [9000, 1, 4097, 6001], seed=3)
    b.check(b.run())
    b.check(b.run(max_kv_len=9000))
    b.check(b.run(window=5000), window=5000)
    # a length bound that is too small costs speed, not tokens; so do large ones
    b.check(b.run(max_kv_len=100, max_q_len=4))
    b.check(b.run(max_kv_len=1 << 20, max_q_len=1000))
    b = Batch(2, 2, 64, 64, 4, 32, [40], [5000], seed=4)
    b.check(b.run())


def test_uniform_rows_without_q_start():
    say("attention uniform")
    for n in (1, 3, 40):
        b = Batch(4, 2, 64, 32, 16, 64, [n] * 3, [n, n + 50, n + 7], seed=n)
        b.check(b.run(uniform=True))
        b.check(b.run(uniform=True, max_q_len=1000))


def test_rows_that_see_nothing_are_zero():
    """More new tokens than cached ones: the first rows have negative positions."""
    say("attention empty rows")
    for n, L in ((5, 3), (100, 40), (1, 0), (300, 0)):
        b = Batch(4, 2, 128, 16, 16, 64, [n, 1], [L, 20], seed=n)
        o = b.run()
        assert not o[:max(0, n - L)].any()
        b.check(o)


def test_large_and_small_scores():
    say("attention scores")
    b = Batch(4, 1, 128, 32, 16, 64, [3, 80], [200, 90], seed=8, spread=30.0)
    b.check(b.run(scale=0.5), scale=0.5)
    b.check(b.run(scale=0.0), scale=0.0)
    b.check(b.run(scale=-0.3), scale=-0.3)
    # all scores hugely negative: the softmax is of their differences
    b = Batch(2, 1, 64, 16, 16, 64, [1, 30], [50, 60], seed=9)
    for x in b.k:
        x[...] = -np.abs(x) * 50
    for x in b.q:
        x[...] = np.abs(x) * 50
    b.fill()
    b.check(b.run(), what="negative scores")


@pytest.mark.parametrize("n", (1, 4, 40, 150))
@pytest.mark.parametrize("D", (64, 128, 256))
def test_values_of_unseen_tokens_stay_out(n, D):
    """Infinities and NaN in a token's key and value reach the rows that see
    it, and no others: later tokens of the chunk, and ones before the window."""
    say(f"attention non-finite n={n} D={D}")
    for window in (0, 33):
        b = Batch(4, 2, D, 32, 16, 64, [n], [n + 90], seed=n)
        last = n + 89
        b.k[0][last], b.v[0][last] = np.nan, np.nan
        if n > 10:
            b.v[0][last - 5] = np.inf
            b.v[0][last - 9, 0, 3] = -np.inf
        hidden = []
        if window:
            for t, val in ((10, np.nan), (3, np.inf), (last - n - window + 1, np.nan)):
                b.k[0][t], b.v[0][t] = val, val
                hidden.append(t)
        b.fill()
        o = b.run(window=window)
        bad = [t for t in range(n + 90) if not (np.isfinite(b.k[0][t]).all() and np.isfinite(b.v[0][t]).all())]
        # the rows' own arithmetic, token by token
        for i in range(n):
            p = 90 + i
            lo = max(0, p - window + 1) if window else 0
            seen = [t for t in bad if lo <= t <= p]
            if not seen:
                ref, w, _ = oracle.decoder.attention(b.q[0][i:i + 1], b.kv[0][0][lo:p + 1], b.kv[1][0][lo:p + 1],
                                                     D ** -0.5)
                err = np.abs(o[i] - ref[0])
                bound = 2.0 ** -11 * np.abs(ref[0]) + (2.0 ** -11 + 2.0 ** -12) * w[0] + 2.0 ** -25 * (1 + (p + 1) * 5)
                assert np.isfinite(o[i]).all() and (err <= bound).all(), (i, err.max())
            elif last in seen:
                assert np.isnan(o[i]).all(), i
            elif n > 10 and last - 5 in seen:
                assert not np.isfinite(o[i]).any(), i
            else:
                c = b.Hq // b.Hk
                assert np.isneginf(o[i][:c, 3]).all(), i
                o2 = np.delete(o[i].reshape(b.Hq, D), 3, axis=1)
                assert np.isfinite(o2).all() and np.isfinite(o[i][c:]).all(), i


def test_strided_queries_and_guards():
    """q as a slice of a fused projection's output; nothing outside out and
    the workspace is written."""
    say("attention strides")
    for n in (1, 50):
        b = Batch(8, 2, 128, 64, 8, 128, [n, n], [300, 170], seed=n)
        dev = device()
        T = 2 * n
        fused = torch.full((T, 8 + 4, 128), float("nan"), dtype=torch.float16, device=dev)
        fused[:, :8] = torch.from_numpy(np.concatenate(b.q)).to(dev)
        need = dq.paged_attention_workspace_bytes(b.cache, T, 8, 2, n, 300)
        ws, og = Guarded(max(need, 16), dev), Guarded(T * 8 * 128 * 2, dev)
        out = og.view(torch.float16, (T, 8, 128))
        o = b.run(q=fused[:, :8], out=out, max_q_len=n, max_kv_len=300, workspace=ws.view(torch.uint8, (max(need, 16),)))
        b.check(o)
        assert ws.intact() and og.intact()


def test_rows_of_no_sequence_are_left_alone():
    say("attention unowned rows")
    b = Batch(4, 2, 64, 32, 16, 64, [3, 2], [20, 30], seed=5)
    dev = device()
    q = torch.zeros((9, 4, 64), dtype=torch.float16, device=dev)
    q[2:7] = torch.from_numpy(np.concatenate(b.q)).to(dev)
    out = torch.full((9, 4, 64), 7.0, dtype=torch.float16, device=dev)
    dq.paged_attention(b.cache, q, torch.from_numpy(b.table).to(dev),
                       torch.tensor(b.kv_lens, dtype=torch.int32, device=dev),
                       torch.tensor([2, 5, 7], dtype=torch.int32, device=dev), out=out)
    torch.cuda.synchronize()
    o = out.float().cpu().numpy().astype(np.float64)
    assert (o[:2] == 7).all() and (o[7:] == 7).all()
    b.check(o[2:7])


def test_repeats_are_bit_equal_and_other_streams_work():
    say("attention streams")
    b = Batch(8, 2, 128, 32, 4, 32, [1, 1, 60], [5000, 40, 200], seed=6)
    o = b.run()
    for _ in range(3):
        assert np.array_equal(o, b.run())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        o2 = b.run()
    assert np.array_equal(o, o2)


def test_graph_replay():
    """A captured call, replayed after its inputs change in place."""
    say("attention graph")
    b = Batch(8, 2, 128, 32, 16, 64, [1, 1], [3000, 64], seed=12)
    dev = device()
    q = torch.from_numpy(np.concatenate(b.q)).to(dev)
    table = torch.from_numpy(b.table).to(dev)
    kv = torch.tensor(b.kv_lens, dtype=torch.int32, device=dev)
    out = torch.zeros((2, 8, 128), dtype=torch.float16, device=dev)
    ws = dq.paged_attention_workspace(b.cache, 2, 8, 2, 1, 3000, dev)
    call = lambda: dq.paged_attention(b.cache, q, table, kv, max_kv_len=3000, out=out, workspace=ws)   # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ((3000, 64), (17, 63), (2999, 1)):
        kv.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got, out)


def test_no_work():
    say("attention no work")
    dev = device()
    c = dq.KVCache.empty(2, 2, 64, page_size=16)
    q = torch.empty((0, 4, 64), dtype=torch.float16, device=dev)
    o = dq.paged_attention(c, q, torch.zeros((0, 1), dtype=torch.int32, device=dev),
                           torch.zeros((0,), dtype=torch.int32, device=dev))
    assert o.shape == (0, 4, 64)


def test_binding_refuses_wrong_tensors():
    dev = device()
    b = Batch(4, 2, 64, 32, 16, 64, [3], [20], seed=5)
    q = torch.zeros((3, 4, 64), dtype=torch.float16, device=dev)
    table = torch.from_numpy(b.table).to(dev)
    kv = torch.tensor([20], dtype=torch.int32, device=dev)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(q=q.transpose(0, 1)), dict(q=q.cpu()),
                dict(block_table=table.long()), dict(kv_len=kv.repeat(2)), dict(q_start=kv),
                dict(out=q[:, :2]), dict(workspace=torch.empty(1 << 20, device=dev))):
        args = dict(q=q, block_table=table, kv_len=kv)
        args.update(bad)
        with pytest.raises(ValueError):
            dq.paged_attention(b.cache, **args)
    with pytest.raises(dq.QlinearError) as e:
        dq.paged_attention(b.cache, q[:, :3].contiguous(), table, kv)
    assert e.value.status == dq._lib.ERR_UNSUPPORTED
    with pytest.raises(dq.QlinearError):
        dq.paged_attention(b.cache, q, table, kv, scale=float("inf"))


@pytest.mark.parametrize("bits,group,D,Hq,Hk", [(16, 64, 64, 8, 2), (4, 32, 64, 4, 4), (8, 64, 128, 8, 1),
                                                (16, 64, 256, 4, 2)])
def test_more_sequences_than_lanes(bits, group, D, Hq, Hk):
    """Batches past 64 and 128 sequences of all kinds: without new tokens,
    without cached ones, with few rows and with many."""
    say(f"attention many sequences bits={bits} D={D}")
    rng = np.random.default_rng(bits + D)
    for B in (64, 65, 150):
        n = rng.choice([0, 1, 1, 1, 2, 5], B)
        L = np.where(rng.random(B) < 0.1, 0, n + rng.integers(0, 90, B))
        n[B - 1], L[B - 1] = 1, 700
        n[3], L[3] = 40, 333
        n[B // 2], L[B // 2] = 2, 450
        b = Batch(Hq, Hk, D, 16, bits, group, n, L, seed=B)
        b.check(b.run(), what=f"B={B}")
        b.check(b.run(window=40, max_kv_len=700), window=40, what=f"B={B}")


@pytest.mark.parametrize("where", (0, 63, 64, 129))
def test_one_long_sequence_among_short_ones(where):
    """Its steps are shared out over workgroups that also have whole sequences."""
    say(f"attention one long at {where}")
    for lens, n in ((1, 1), (40, 1), (0, 1), (9, 3)):
        L = [lens] * 130
        L[where] = 6000
        b = Batch(4, 2, 64, 64, 16, 64, [n] * 130, L, seed=where)
        b.check(b.run(), what=f"lens={lens}")


@pytest.mark.parametrize("D,bits", [(64, 16), (128, 16), (128, 4), (256, 8)])
def test_drafts_over_long_caches(D, bits):
    """One to four row tiles per sequence, lengths off the step, tile and span edges."""
    say(f"attention drafts D={D} bits={bits}")
    for Hq, n in ((8, 2), (8, 3), (8, 4), (8, 5), (8, 8), (16, 4), (5, 7)):
        b = Batch(Hq, 1, D, 32, bits, 64, [n] * 5, [2049, 700, 3001, n, 1500], seed=Hq + n)
        b.check(b.run(), what=f"{Hq} heads, {n} tokens")
        b.check(b.run(window=900), window=900, what=f"{Hq} heads, {n} tokens")


@pytest.mark.parametrize("n", (1, 6, 130))
@pytest.mark.parametrize("bits", (8, 6, 4))
def test_unseen_quantized_nan_stays_out(n, bits):
    """A quantized row of NaN has a NaN scale: the rows that see it are NaN, the others untouched."""
    say(f"attention NaN scales n={n} bits={bits}")
    window = 50
    b = Batch(4, 2, 128, 32, bits, 32, [n], [n + 400], seed=n + bits)
    hidden, last = 400 - window + 1, n + 399       # the first is seen by row 0 alone, one more by none
    for t in (hidden - 1, hidden, last):
        b.k[0][t] = b.v[0][t] = np.nan
    b.fill()
    o = b.run(window=window)
    for i in range(n):
        p = 400 + i
        lo = p - window + 1
        if lo <= hidden or p == last:
            assert np.isnan(o[i]).all(), i
            continue
        ref, w, _ = oracle.decoder.attention(b.q[0][i:i + 1], b.kv[0][0][lo:p + 1], b.kv[1][0][lo:p + 1], 128 ** -0.5)
        bound = 2.0 ** -11 * np.abs(ref[0]) + (2.0 ** -11 + 2.0 ** -12) * w[0] + 2.0 ** -25 * (1 + (p + 1) * 5)
        assert np.isfinite(o[i]).all() and (np.abs(o[i] - ref[0]) <= bound).all(), i


@pytest.mark.parametrize("D,bits,Hq,Hk", [(128, 16, 8, 8), (64, 4, 16, 8), (256, 8, 8, 8)])
def test_batches_of_near_equal_lengths(D, bits, Hq, Hk):
    """Fewer and more tiles than the chip holds workgroups of a head, in lengths
    near one another, with one much longer, and with some sequences without new tokens."""
    say(f"attention near-equal lengths D={D} bits={bits}")
    rng = np.random.default_rng(D + bits)
    for B, n in ((2, 1), (20, 2), (65, 1)):
        L = rng.integers(560, 640, B)
        q = np.full(B, n)
        b = Batch(Hq, Hk, D, 64, bits, 64, q, L, seed=B)
        b.check(b.run(), what=f"B={B}")
        q[B // 2], L[B // 3] = 0, 2500
        b = Batch(Hq, Hk, D, 64, bits, 64, q, L, seed=B + 1)
        b.check(b.run(), what=f"B={B}, one long")


@pytest.mark.parametrize("n", (1, 100))
def test_pools_past_32_bit_offsets(n):
    """Appended to, copied within and read from pages that lie more than 2^32 bytes and elements into a pool."""
    say(f"attention large pool n={n}")
    dev = device()
    D, P, Hk, pages = 128, 64, 2, 270000       # 2^32 elements of a pool are 262144 pages
    cache = dq.KVCache.empty(pages, Hk, D, page_size=P)
    rng = np.random.default_rng(n)
    L = 150
    q, k, v = (rng.standard_normal((m, h, D)).astype(np.float16) for m, h in ((n, 4), (L, Hk), (L, Hk)))
    held, first = [269999, 131073, 262145], [269990, 131070, 262140]
    slots = [first[t // P] * P + t % P for t in range(L)]
    dq.rope_append(cache, None, torch.from_numpy(k).to(dev), torch.from_numpy(v).to(dev), None,
                   torch.tensor(slots, dtype=torch.int32, device=dev), None)
    dq.copy_pages([cache], torch.tensor(list(zip(first, held)), dtype=torch.int32, device=dev))
    o = dq.paged_attention(cache, torch.from_numpy(q).to(dev), torch.tensor([held], dtype=torch.int32, device=dev),
                           torch.tensor([L], dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    ref, w, total = oracle.decoder.attention(q, k.astype(np.float64), v.astype(np.float64), D ** -0.5)
    err = np.abs(o.double().cpu().numpy() - ref)
    tiny = L * np.abs(v).max() / np.maximum(total, 1.0)
    assert (err <= 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -12) * w + 2.0 ** -25 * (1 + tiny[..., None])).all()


@pytest.mark.parametrize("D", (64, 128, 256))
def test_long_chunks_from_memory(D):
    """Many whole steps, rows staged from memory rather than from a cache, one
    range of steps and several: no step may use rows that have not arrived."""
    say(f"attention long chunk D={D}")
    n, past = 150, 5000
    b = Batch(4, 2, D, 64, 16, 64, [n], [n + past], seed=D)
    ref, w, total = oracle.decoder.attention(b.q[0], b.kv[0][0], b.kv[1][0], D ** -0.5)
    tiny = (n + past) * np.abs(b.kv[1][0]).max() / np.maximum(total, 1.0)
    bound = 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -12) * w + 2.0 ** -25 * (1 + tiny[..., None])
    other = torch.empty(1 << 30, dtype=torch.uint8, device=device())
    # a small length bound plans one range
    assert dq.paged_attention_workspace_bytes(b.cache, n, 4, 1, n, n + past) > 0
    for kw in (dict(max_kv_len=n), dict(max_kv_len=n + past)):
        for _ in range(3):
            other.add_(1)          # what the caches hold now
            o = b.run(**kw)
            assert (np.abs(o - ref) <= bound).all(), (kw, (np.abs(o - ref) / bound).max())


@pytest.mark.parametrize("n,L", [(5, 3), (100, 40), (3, 0)])
def test_windows_that_end_nowhere(n, L):
    """The largest windows hide nothing, also from rows before the first token."""
    say(f"attention window 2^31 - 1 n={n} L={L}")
    for D in (64, 128):
        b = Batch(4, 2, D, 16, 16, 64, [n, 1], [L, 700], seed=n)
        for window in (2 ** 31 - 1, 2 ** 31 - n):
            b.check(b.run(window=window), what=f"window={window}")


@pytest.mark.parametrize("n", (3, 150))
@pytest.mark.parametrize("value", (np.nan, np.inf))
def test_non_finite_queries(n, value):
    """A NaN or infinity in a head's query makes that row NaN (its scores are, or
    their differences), at any scale, zero among them, and leaves the others."""
    say(f"attention non-finite query n={n} {value}")
    b = Batch(4, 2, 64, 32, 16, 64, [n], [n + 90], seed=n)
    b.q[0][1, 2, 5] = b.q[0][n - 1, 3, 63] = value
    hit = np.zeros((n, 4), bool)
    hit[1, 2] = hit[n - 1, 3] = True
    finite = np.where(hit[..., None], 0, b.q[0])
    for scale in (0.0, 0.1, -0.1):
        o = b.run(scale=scale)
        ref, w, total = oracle.decoder.attention(finite, b.kv[0][0], b.kv[1][0], scale)
        tiny = (n + 90) * np.abs(b.kv[1][0]).max() / np.maximum(total, 1.0)
        bound = 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -12) * w + 2.0 ** -25 * (1 + tiny[..., None])
        assert np.isnan(o[hit]).all(), scale
        assert (np.abs(o - ref)[~hit] <= bound[~hit]).all(), scale


def test_sizes_past_32_bits():
    say("attention sizes past 32 bits")
    b = Batch(4, 2, 64, 32, 16, 64, [3, 70], [200, 90], seed=3)
    o = b.run()
    for kw in (dict(window=2 ** 32 + 1), dict(max_kv_len=2 ** 32 + 1), dict(max_q_len=2 ** 32 + 1)):
        assert np.array_equal(b.run(**kw), o), kw
    with pytest.raises(dq.QlinearError):
        b.run(window=1 - 2 ** 32)


def test_one_workspace_for_the_chunks_of_a_prompt():
    say("attention workspace")
    dev = device()
    top = 700
    cache = None
    for n, past in ((top, 0), (300, 4000), (33, 9000), (3, 9000), (1, 9000)):
        b = Batch(8, 2, 64, 64, 16, 64, [n], [n + past], seed=n)
        if cache is None:
            cache = b.cache
            ws = dq.paged_attention_workspace(cache, top, 8, 1, top, 10000, dev)
        b.check(b.run(max_q_len=n, max_kv_len=10000, workspace=ws), what=f"n={n}")
