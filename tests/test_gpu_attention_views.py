"""Attention with sinks and over shared prefixes against the float64 oracle.

The error bound is that of paged attention (see test_gpu_attention.py): results
of parts of a row are joined in float32, whose factors are at most 1, so that
what each part adds to the error is what the same tokens add in one.
"""

import numpy as np
import pytest
import torch

import dequant_matmul_gptq_amd as dq
import oracle
from gpu_util import Guarded, device, say
from test_gpu_attention import Batch

pytestmark = pytest.mark.gpu


def _close(b, i, got, ref, w, total, what):
    vmax = np.abs(b.kv[1][i]).max() if b.kv_lens[i] else 0.0
    tiny = b.kv_lens[i] * vmax / np.maximum(total, 1.0)
    bound = 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -12) * w + 2.0 ** -25 * (1 + tiny[..., None])
    assert np.isfinite(got).all(), f"{what} sequence {i}: non-finite output"
    err = np.abs(got - ref)
    assert (err <= bound).all(), f"{what} sequence {i}: error {err.max():.3e}, {(err / bound).max():.2f} bounds"


# ---------------------------------------------------------------- sinks

def _check_sinks(b, window, sinks, what="", **kw):
    """The call, with NaN in all tokens that no new one sees."""
    for i, (n, L) in enumerate(zip(b.q_lens, b.kv_lens)):
        for t in range(sinks, max(0, L - n - window + 1)):
            b.k[i][t] = b.v[i][t] = np.nan
    b.fill()
    o = b.run(window=window, sinks=sinks, **kw)
    at = 0
    for i, n in enumerate(b.q_lens):
        L = b.kv_lens[i]
        k, v = (np.nan_to_num(x[i], nan=0.0) for x in b.kv)
        ref, w, total = oracle.decoder.attention(b.q[i], k, v, b.D ** -0.5, window, sinks)
        b.kv[1][i] = v
        _close(b, i, o[at:at + n], ref, w, total, f"{what} window={window} sinks={sinks}")
        at += n
    return o


PAIRS = [(1, 1), (16, 1), (20, 4), (33, 31), (33, 32), (64, 33), (50, 64), (5, 100), (100, 300), (200, 2 ** 31 - 1),
         (2 ** 31 - 1, 4)]


@pytest.mark.parametrize("bits,group", [(16, 128), (8, 64), (6, 32), (4, 128)])
@pytest.mark.parametrize("window,sinks", PAIRS)
def test_sinks_single_tokens(bits, group, window, sinks):
    say(f"sinks decode bits={bits} window={window} sinks={sinks}")
    b = Batch(8, 2, 128, 32, bits, group, [1] * 9, [1, 2, 17, 33, 70, 129, 257, 700, 300], seed=bits + sinks % 97)
    _check_sinks(b, window, sinks)


@pytest.mark.parametrize("D,bits", [(64, 16), (64, 8), (64, 6), (64, 4), (128, 16), (128, 4), (256, 16), (256, 6)])
@pytest.mark.parametrize("n,past", [(2, 200), (7, 300), (33, 5), (64, 500), (65, 63), (150, 700), (300, 0)])
@pytest.mark.parametrize("window,sinks", [(1, 4), (40, 1), (50, 64), (70, 130), (129, 33)])
def test_sinks_chunks(D, bits, n, past, window, sinks):
    say(f"sinks chunk n={n} past={past} D={D} bits={bits} window={window} sinks={sinks}")
    b = Batch(4, 2, D, 32, bits, 64, [n], [n + past], seed=n + past + bits)
    _check_sinks(b, window, sinks)


@pytest.mark.parametrize("Hq,Hk", [(4, 4), (8, 1), (6, 2), (20, 4), (33, 1)])
@pytest.mark.parametrize("D", (64, 128, 256))
def test_sinks_head_layouts(Hq, Hk, D):
    say(f"sinks heads {Hq}/{Hk} D={D}")
    b = Batch(Hq, Hk, D, 64, 16, 64, [1, 3, 40, 1], [165, 230, 340, 7], seed=Hq + D)
    _check_sinks(b, 60, 10)


@pytest.mark.parametrize("bits", (16, 4))
def test_sinks_long_and_mixed(bits):
    """Spans that start and end among the sinks, in the window and past it."""
    say(f"sinks long bits={bits}")
    b = Batch(4, 1, 128, 256, bits, 128, [1, 1, 4, 1, 200, 0, 1], [9000, 1, 6001, 4097, 3000, 50, 0], seed=3)
    _check_sinks(b, 2000, 300)
    _check_sinks(b, 700, 64)
    b = Batch(8, 8, 128, 16, bits, 32, [1] * 70, [1 + 37 * i for i in range(70)], seed=4)
    _check_sinks(b, 900, 5)


@pytest.mark.parametrize("bits,group", [(16, 128), (8, 64), (6, 32), (4, 128)])
@pytest.mark.parametrize("D", (64, 128, 256))
@pytest.mark.parametrize("n,window,sinks", [(7, 23, 1), (8, 5, 33), (6, 40, 100), (2, 1, 2)])
def test_sinks_of_tiles_that_start_behind_them(D, bits, group, n, window, sinks):
    """Rows of a sequence in several tiles, whose windows start in other steps than its first row's, with sinks
    before, in and behind that step."""
    say(f"sinks tiles D={D} bits={bits} n={n} window={window} sinks={sinks}")
    lens = [n, 33, 35, 60, 64, 66, 79, 91, 97, 130, 342]
    for Hq, Hk in ((16, 2), (8, 4)):
        b = Batch(Hq, Hk, D, 128, bits, min(group, D), [n] * len(lens), lens, seed=D + bits + n)
        _check_sinks(b, window, sinks)


def test_sinks_without_a_window_and_bounds():
    say("sinks bounds")
    b = Batch(8, 2, 64, 16, 16, 64, [1, 30], [700, 90], seed=5)
    b.check(b.run(sinks=9), what="no window")
    assert np.array_equal(b.run(window=40, sinks=0), b.run(window=40))
    o = b.run(window=40, sinks=7)
    for kw in (dict(max_kv_len=10), dict(max_kv_len=1 << 20, max_q_len=1000)):
        got = b.run(window=40, sinks=7, **kw)
        assert np.abs(got - o).max() < 2e-3
    _check_sinks(Batch(4, 2, 64, 32, 16, 64, [40] * 3, [400, 90, 47], seed=6), 30, 5, uniform=True)


@pytest.mark.parametrize("n", (1, 4, 40, 150))
@pytest.mark.parametrize("D", (64, 128, 256))
def test_sinks_values_reach_the_rows_that_see_them(n, D):
    """An infinity among the sinks reaches every row, one in the window those that see it."""
    say(f"sinks non-finite n={n} D={D}")
    window, sinks, L = 33, 40, n + 200
    b = Batch(4, 2, D, 32, 16, 64, [n], [L], seed=n)
    first = L - n - window + 1
    b.v[0][first, 0, 3] = np.inf          # the first row's window starts with it
    b.fill()
    o = b.run(window=window, sinks=sinks).reshape(n, 4, D)
    seen = np.zeros((n, 4, D), bool)
    seen[0, :2, 3] = True
    assert np.isposinf(o[seen]).all() and np.isfinite(o[~seen]).all()
    b.v[0][first, 0, 3] = 0
    b.v[0][sinks - 1, 1, 5] = -np.inf
    b.fill()
    o = b.run(window=window, sinks=sinks).reshape(n, 4, D)
    seen[:] = False
    seen[:, 2:, 5] = True
    assert np.isneginf(o[seen]).all() and np.isfinite(o[~seen]).all()


def test_sinks_graph_streams_and_workspace():
    say("sinks graph")
    b = Batch(8, 2, 128, 32, 16, 64, [1, 1], [3000, 64], seed=12)
    dev = device()
    q = torch.from_numpy(np.concatenate(b.q)).to(dev)
    table = torch.from_numpy(b.table).to(dev)
    kv = torch.tensor(b.kv_lens, dtype=torch.int32, device=dev)
    out = torch.zeros((2, 8, 128), dtype=torch.float16, device=dev)
    need = dq.paged_attention_workspace_bytes(b.cache, 2, 8, 2, 1, 3000, 1000, 50)
    ws = Guarded(max(need, 16), dev)
    call = lambda: dq.paged_attention(b.cache, q, table, kv, max_kv_len=3000, out=out, workspace=ws.bytes(),    # noqa: E731
                                      window=1000, sinks=50)
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
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            want = dq.paged_attention(b.cache, q, table, kv, max_kv_len=3000, window=1000, sinks=50)
        s.synchronize()
        assert torch.equal(got, want) and ws.intact()


# ---------------------------------------------------------------- shared prefixes

class Shared(Batch):
    """Groups of sequences with common first tokens; each group's full pages are
    shared, and what other sequences than its first have in the block table
    below the shared length is no page. Sequences past the groups share nothing."""

    def __init__(self, Hq, Hk, D, P, bits, group, sizes, shared, q_lens, tails, seed=0, gap=0):
        """sizes, shared: of the groups; tails: each sequence's tokens after the shared ones; gap: sequences
        before the first group."""
        rng = np.random.default_rng(seed)
        self.Hq, self.Hk, self.D, self.P, self.bits, self.group = Hq, Hk, D, P, bits, group
        self.sizes, self.shared = list(sizes), list(shared)
        self.starts = [gap + sum(sizes[:i]) for i in range(len(sizes) + 1)]
        low = [0] * len(tails)
        of = [None] * len(tails)
        for g, s in enumerate(shared):
            for i in range(self.starts[g], self.starts[g + 1]):
                low[i], of[i] = s, g
        self.low, self.q_lens = low, list(q_lens)
        self.kv_lens = [s + t for s, t in zip(low, tails)]
        heads = [[rng.standard_normal((s, Hk, D)).astype(np.float16) for s in shared] for _ in range(2)]
        scale = rng.uniform(0.5, 1.5, D)
        self.q = [rng.standard_normal((n, Hq, D)).astype(np.float16) for n in q_lens]
        self.k, self.v = [], []
        for i, t in enumerate(tails):
            k, v = (rng.standard_normal((t, Hk, D)).astype(np.float16) for _ in range(2))
            none = np.zeros((0, Hk, D), np.float16)
            self.k.append((np.concatenate([none if of[i] is None else heads[0][of[i]], k]) * scale).astype(np.float16))
            self.v.append(np.concatenate([none if of[i] is None else heads[1][of[i]], v]))
        need = [-(-L // P) for L in self.kv_lens]
        full = [s // P for s in low]
        self.pages = sum(need) + 2
        order = list(rng.permutation(self.pages))
        self.table = np.full((len(tails), max(need + [1]) + 1), -7, np.int32)
        for i in range(len(tails)):
            first = of[i] is None or i == self.starts[of[i]]
            if not first:
                self.table[i, :full[i]] = self.table[self.starts[of[i]], :full[i]]
            for p in range(0 if first else full[i], need[i]):
                self.table[i, p] = order.pop()
        self.fill()
        self.call_table = self.table.copy()
        for i in range(len(tails)):
            if of[i] is not None and i != self.starts[of[i]]:
                self.call_table[i, :full[i]] = -9

    def call(self, uniform=False, one=False, q=None, **kw):
        dev = device()
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
        qt = torch.from_numpy(np.concatenate(self.q)).to(dev) if q is None else q
        starts = None if uniform else ints(np.concatenate([[0], np.cumsum(self.q_lens)]))
        o = dq.paged_attention_shared(self.cache, qt, ints(self.call_table), ints(self.kv_lens), ints(self.shared),
                                      None if one else ints(self.starts), starts, **kw)
        torch.cuda.synchronize()
        return o.float().cpu().numpy().astype(np.float64)

    def compare(self, o, what="", scale=None):
        at = 0
        for i, n in enumerate(self.q_lens):
            ref, w, total = oracle.decoder.attention(self.q[i], self.kv[0][i], self.kv[1][i],
                                                     self.D ** -0.5 if scale is None else scale)
            _close(self, i, o[at:at + n], ref, w, total, what)
            at += n


@pytest.mark.parametrize("bits,group", [(16, 128), (8, 64), (6, 32), (4, 128)])
@pytest.mark.parametrize("P", (16, 256))
@pytest.mark.parametrize("shared", (1, 31, 32, 33, 256, 1000))
def test_shared_single_tokens(bits, group, P, shared):
    """Lengths of the prefix inside pages and steps; up to 16 rows a key/value head together."""
    say(f"shared decode bits={bits} P={P} shared={shared}")
    b = Shared(8, 2, 128, P, bits, group, [4], [shared], [1] * 4, [1, 2, 40, 300], seed=bits + P + shared)
    b.compare(b.call())
    b.compare(b.call(one=True, max_q_len=1, max_kv_len=1300, max_shared_len=shared))
    b.compare(b.call(uniform=True))


@pytest.mark.parametrize("Hq,Hk", [(4, 4), (8, 1), (6, 2), (16, 1), (20, 4), (33, 1), (64, 8)])
@pytest.mark.parametrize("D", (64, 128, 256))
@pytest.mark.parametrize("count", (1, 3, 17, 40))
def test_shared_head_layouts(Hq, Hk, D, count):
    """One to 40 sequences: prefixes in the few-row kernel's tiles and in the other's."""
    say(f"shared heads {Hq}/{Hk} D={D} count={count}")
    for bits, P in ((16, 32), (4, 64)):
        b = Shared(Hq, Hk, D, P, bits, 64, [count], [130], [1 + i % 2 for i in range(count)],
                   [2 + 7 * i % 90 for i in range(count)], seed=Hq + D + count)
        b.compare(b.call(), f"bits={bits}")


@pytest.mark.parametrize("bits", (16, 8, 4))
def test_shared_groups(bits):
    """Groups of many sizes, one of a single sequence, one that shares nothing, sequences of no group before and
    after them, prompts, drafts and single tokens, sequences without new tokens or without any."""
    say(f"shared groups bits={bits}")
    b = Shared(8, 2, 64, 16, bits, 32, [3, 1, 0, 2, 4], [100, 333, 50, 0, 17],
               [2, 1, 3, 70, 1, 5, 1, 0, 1, 130, 0, 1, 1], [40, 1, 3, 99, 300, 5, 1, 7, 90, 140, 0, 600, 1], seed=bits, gap=1)
    b.compare(b.call())
    b.compare(b.call(max_q_len=130, max_kv_len=800, max_shared_len=333))
    b.compare(b.call(max_q_len=130, max_kv_len=100, max_shared_len=1))        # too small bounds cost speed


def test_shared_long():
    """Prefixes and own tokens that are cut over workgroups by both kernels."""
    say("shared long")
    for bits, Hq, Hk, n, count in ((16, 8, 1, 1, 6), (16, 8, 1, 1, 40), (4, 16, 4, 4, 20), (8, 2, 2, 1, 5)):
        b = Shared(Hq, Hk, 128, 256, bits, 128, [count], [9000], [n] * count, [n + 400 * (i % 3) for i in range(count)], seed=count)
        b.compare(b.call(max_q_len=n, max_kv_len=9900, max_shared_len=9000), f"bits={bits} {Hq}/{Hk} x{count}")
    b = Shared(4, 1, 64, 64, 16, 64, [2, 3], [5000, 3000], [1] * 6, [900, 1, 20, 3000, 5, 6000], seed=9)
    b.compare(b.call())


@pytest.mark.parametrize("D,bits", [(64, 16), (128, 16), (128, 8), (256, 16), (256, 4)])
def test_shared_prompts(D, bits):
    say(f"shared prompts D={D} bits={bits}")
    b = Shared(8, 2, D, 32, bits, 64, [3, 2], [700, 130], [150, 41, 200, 90, 300], [150, 41, 260, 90, 333], seed=D)
    b.compare(b.call())
    b = Shared(8, 2, D, 32, bits, 64, [2], [2100], [40, 30], [40, 30], seed=D + 1)
    b.compare(b.call(max_q_len=40, max_kv_len=2140, max_shared_len=2100))


def test_shared_many_sequences():
    say("shared many")
    b = Shared(4, 1, 64, 16, 16, 64, [100, 30], [64, 48], [1] * 140, [1 + i % 50 for i in range(140)], seed=2)
    b.compare(b.call())
    b = Shared(4, 1, 64, 16, 16, 64, [2] * 70, [16 + i for i in range(70)], [1] * 140, [1 + i % 50 for i in range(140)], seed=3)
    b.compare(b.call())


@pytest.mark.parametrize("bits", (16, 6))
def test_shared_prompt_among_many(bits):
    """A prompt among so many single tokens that the bound on row tiles is past what the chip holds, and the tiles
    themselves are not."""
    say(f"shared prompt among many bits={bits}")
    n = [1] * 30 + [40] + [1] * 59
    b = Shared(32, 8, 64, 64, bits, 32, [70, 20], [900, 400], n, [x + 9 * i % 80 for i, x in enumerate(n)], seed=bits)
    b.compare(b.call())


def test_shared_rows_that_see_nothing_of_their_own():
    """More new tokens than own ones: nothing is shared there, and the first rows have no position."""
    say("shared empty")
    b = Shared(4, 2, 64, 16, 16, 64, [2], [0], [5, 3], [3, 0], seed=4)
    o = b.call()
    assert not o[:2].any() and not o[5:].any()
    b.compare(o)
    # the prefix alone is seen where the own tokens say nothing (shared_len == kv_len - n would show one more)
    b = Shared(4, 2, 64, 16, 16, 64, [2], [50], [1, 1], [1, 1], seed=5)
    b.compare(b.call())


def test_shared_scores_and_scales():
    say("shared scores")
    b = Shared(4, 1, 128, 32, 16, 64, [3], [200], [1, 70, 2], [20, 90, 3], seed=8)
    for x in b.q:
        x *= 30
    for scale in (0.5, 0.0, -0.3):
        b.compare(b.call(scale=scale), f"scale={scale}", scale=scale)
    # own tokens that outweigh the prefix by far, and the other way
    for own in (60.0, -60.0):
        b = Shared(4, 1, 64, 32, 16, 64, [2], [100], [1, 2], [30, 40], seed=9)
        for i in range(2):
            b.q[i][...] = np.abs(b.q[i])
            b.k[i][:100] = 0.5
            b.k[i][100:] = own
        b.fill()
        b.compare(b.call(), f"own={own}")


@pytest.mark.parametrize("count", (3, 30))
def test_shared_values_of_other_sequences_stay_out(count):
    """NaN in one sequence's own tokens reaches its rows alone, an infinity in the prefix all rows of the group."""
    say(f"shared non-finite count={count}")
    b = Shared(8, 2, 128, 32, 16, 64, [count, 2], [100, 70], [1] * (count + 2), [20 + i for i in range(count + 2)], seed=count)
    b.v[1][110] = np.nan
    b.fill()
    o = b.call()
    bad = ~np.isfinite(o).reshape(count + 2, -1)
    assert bad[1].all() and not bad[[i for i in range(count + 2) if i != 1]].any()
    b.v[1][110] = 1
    for i in range(count):
        b.v[i][7, 0, 3] = np.inf
    b.fill()
    o = b.call().reshape(count + 2, 8, 128)
    seen = np.zeros(o.shape, bool)
    seen[:count, :4, 3] = True
    assert np.isposinf(o[seen]).all() and np.isfinite(o[~seen]).all()


def test_shared_rows_of_no_sequence_strides_and_guards():
    say("shared guards")
    for n, count in ((1, 3), (40, 3), (1, 30)):
        b = Shared(8, 2, 128, 64, 8, 128, [count], [300], [n] * count, [n + i for i in range(count)], seed=n)
        dev = device()
        T = n * count + 5
        fused = torch.full((T, 8 + 4, 128), float("nan"), dtype=torch.float16, device=dev)
        fused[2:T - 3, :8] = torch.from_numpy(np.concatenate(b.q)).to(dev)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
        need = dq.paged_attention_shared_workspace_bytes(b.cache, T, 8, count, n, 400, 1, 300)
        ws, og = Guarded(need, dev), Guarded(T * 8 * 128 * 2, dev)
        out = og.view(torch.float16, (T, 8, 128))
        out.fill_(7)
        dq.paged_attention_shared(b.cache, fused[:, :8], ints(b.call_table), ints(b.kv_lens), ints([300]), None,
                                  ints([2 + n * i for i in range(count + 1)]), max_q_len=n, max_kv_len=400,
                                  max_shared_len=300, out=out, workspace=ws.bytes())
        assert ws.intact() and og.intact()
        o = out.float().cpu().numpy().astype(np.float64)
        assert (o[:2] == 7).all() and (o[T - 3:] == 7).all()
        b.compare(o[2:T - 3])


def test_sinks_rows_of_no_sequence_strides_and_guards():
    """Spans that are joined, prompts beside them, rows before the first sequence and behind the last."""
    say("sinks guards")
    for bits, lens, n in ((16, [3000, 700, 2000], [1, 4, 1]), (8, [5000, 300, 90], [2, 1, 40])):
        b = Batch(8, 2, 128, 64, bits, 128, n, lens, seed=bits)
        dev = device()
        T = sum(n) + 5
        fused = torch.full((T, 8 + 4, 128), float("nan"), dtype=torch.float16, device=dev)
        fused[2:T - 3, :8] = torch.from_numpy(np.concatenate(b.q)).to(dev)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
        need = dq.paged_attention_workspace_bytes(b.cache, T, 8, 3, max(n), max(lens), 1500, 40)
        assert need > 0
        ws, og = Guarded(need, dev), Guarded(T * 8 * 128 * 2, dev)
        out = og.view(torch.float16, (T, 8, 128))
        out.fill_(7)
        dq.paged_attention(b.cache, fused[:, :8], ints(b.table), ints(lens), ints(np.cumsum([2] + n)), max(n), max(lens),
                           window=1500, out=out, workspace=ws.bytes(), sinks=40)
        assert ws.intact() and og.intact()
        o = out.float().cpu().numpy().astype(np.float64)
        assert (o[:2] == 7).all() and (o[T - 3:] == 7).all()
        at = 2
        for i, m in enumerate(n):
            ref, w, total = oracle.decoder.attention(b.q[i], b.kv[0][i], b.kv[1][i], 128 ** -0.5, 1500, 40)
            _close(b, i, o[at:at + m], ref, w, total, f"bits={bits}")
            at += m


def test_shared_one_workspace_for_two_graphs():
    """Calls of two sizes, captured with one workspace, replayed in turn."""
    say("shared two graphs")
    dev = device()
    one = Shared(8, 2, 128, 32, 16, 64, [5, 2], [900, 64], [1] * 7, [1 + 50 * i for i in range(7)], seed=13)
    two = Shared(8, 2, 128, 32, 16, 64, [30], [1500], [2] * 30, [2 + 9 * i for i in range(30)], seed=14)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
    ws = dq.paged_attention_shared_workspace(two.cache, 60, 8, 30, 2, 2000, 2, 1500, dev)
    calls = []
    for b, n in ((one, 1), (two, 2)):
        q = torch.from_numpy(np.concatenate(b.q)).to(dev)
        where = [ints(b.table), ints(b.kv_lens), ints(b.shared), ints(b.starts),
                 ints(np.concatenate([[0], np.cumsum(b.q_lens)]))]
        out = torch.zeros(q.shape, dtype=torch.float16, device=dev)

        def call(b=b, q=q, where=where, out=out, n=n):
            dq.paged_attention_shared(b.cache, q, *where, max_q_len=n, max_kv_len=2000, max_shared_len=max(b.shared),
                                      out=out, workspace=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        calls.append((g, b, out))
    for _ in range(3):
        for g, b, out in calls:
            out.fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            b.compare(out.float().cpu().numpy().astype(np.float64))


def test_shared_graph_streams_and_repeats():
    say("shared graph")
    b = Shared(8, 2, 128, 32, 16, 64, [5, 2], [900, 64], [1] * 7, [1 + 50 * i for i in range(7)], seed=12)
    dev = device()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
    q = torch.from_numpy(np.concatenate(b.q)).to(dev)
    table, kv, shared, starts = ints(b.table), ints(b.kv_lens), ints(b.shared), ints(b.starts)
    out = torch.zeros((7, 8, 128), dtype=torch.float16, device=dev)
    ws = dq.paged_attention_shared_workspace(b.cache, 7, 8, 7, 1, 1300, 2, 900, dev)
    call = lambda w=ws, o=out: dq.paged_attention_shared(b.cache, q, table, kv, shared, starts, max_q_len=1, max_kv_len=1300,    # noqa: E731
                                                         max_shared_len=900, out=o, workspace=w)
    call()
    torch.cuda.synchronize()
    b.compare(out.float().cpu().numpy().astype(np.float64))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens, own in (((900, 64), 0), ((320, 32), 0), ((0, 64), 0), ((900, 64), 1)):
        shared.copy_(torch.tensor(lens, dtype=torch.int32))
        kv.copy_(torch.tensor([max(1, L - own) if i else L for i, L in enumerate(b.kv_lens)], dtype=torch.int32))
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            want = call(None, None)
        s.synchronize()
        assert torch.equal(got, want)


def test_shared_equals_plain_attention_of_forks():
    """Pages forked by the pool, as a server has them: the same result as without sharing, to rounding."""
    say("shared forks")
    dev = device()
    rng = np.random.default_rng(1)
    pool, cache = dq.PagePool(64, 16), dq.KVCache.empty(64, 2, 64, page_size=16)
    table = dq.rope_table(512, 64).to(dev)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731

    def append(seq, n):
        at = pool.length(seq)
        slots = pool.extend(seq, n)
        k, v = (torch.from_numpy(rng.standard_normal((n, 2, 64)).astype(np.float16)).to(dev) for _ in range(2))
        dq.rope_append(cache, None, k, v, ints(list(range(at, at + n))), ints(slots), table)

    pool.add("a")
    append("a", 75)
    for name in "bcd":
        pairs = pool.fork("a", name)
        dq.copy_pages([cache], ints(pairs))
    shared = pool.shared_tokens("abcd")
    assert shared == 64
    for i, name in enumerate("abcd"):
        append(name, 1 + 9 * i)
    pages = [pool.pages(s) for s in "abcd"]
    width = max(map(len, pages))
    q = torch.from_numpy(rng.standard_normal((4, 8, 64)).astype(np.float16)).to(dev)
    bt, kv = ints([p + [0] * (width - len(p)) for p in pages]), ints([pool.length(s) for s in "abcd"])
    a = dq.paged_attention(cache, q, bt, kv)
    b = dq.paged_attention_shared(cache, q, bt, kv, ints([shared]))
    assert (a.float() - b.float()).abs().max().item() < 2e-3
