"""A decoder with quantized layers and a paged key/value cache, serving
sequences that come, share a prompt, branch and go: the library's calls in the
order in which a server makes them. Weights are random.

    python examples/decoder.py [--layers 4] [--hidden 4096] [--heads 32] [--kv-heads 8] [--bits 16]

prints the times of a prompt, of single-token steps over four branches of it,
and the pages that the branches share.
"""

from __future__ import annotations

import argparse
import math
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dequant_matmul_gptq_amd as dq  # noqa: E402


class Linear:
    """A 4-bit matrix [K][N] with one float16 scale per 64 rows and column."""

    GROUP = 64

    def __init__(self, K: int, N: int, gen: torch.Generator):
        dev = gen.device
        self.layout = dq.Layout(K, N, self.GROUP, [4] * (K // self.GROUP))
        self.codes = torch.randint(0, 16, (K, N), dtype=torch.uint8, device=dev, generator=gen)
        self.qweight = dq.pack_weights(self.layout, self.codes)
        # codes spread evenly over -8 .. 7 have a variance of 21: this keeps x's scale
        self.scales = torch.full((K // self.GROUP, N), 1.0 / math.sqrt(21.25 * K), dtype=torch.float16, device=dev)
        self.workspace = dq.qgemv_workspace(self.layout, dev)

    def __call__(self, x: torch.Tensor, activation: int = dq.ACT_NONE) -> torch.Tensor:
        if x.shape[0] <= dq.GEMV_MAX_M:
            return dq.qgemv(self.layout, x, self.qweight, self.scales, None, None, self.workspace,
                            activation=activation)
        return dq.qgemm(self.layout, x, self.qweight, self.scales, None, None, activation=activation)


class Decoder:
    """layers of: norm, q/k/v, rotary step into the cache, attention, output
    projection, norm, gated MLP. A step takes any mix of sequences, each with
    its new tokens: whole prompts, parts of them, drafts, single tokens."""

    def __init__(self, layers: int = 4, hidden: int = 4096, heads: int = 32, kv_heads: int = 8, mlp: int = 11008,
                 vocab: int = 32000, pages: int = 256, page_size: int = 64, max_pos: int = 8192, bits: int = 16,
                 window: int = 0, seed: int = 0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        D = hidden // heads
        self.heads, self.kv_heads, self.dim, self.window, self.device = heads, kv_heads, D, window, torch.device(device)
        self.embedding = torch.randn((vocab, hidden), generator=gen, device=device).half()
        self.table = dq.rope_table(max_pos, D, device=device)
        self.layers = []
        for _ in range(layers):
            norms = [(1 + 0.1 * torch.randn(hidden, generator=gen, device=device)).half() for _ in range(2)]
            self.layers.append(dict(
                norms=norms, qkv=Linear(hidden, (heads + 2 * kv_heads) * D, gen), out=Linear(hidden, hidden, gen),
                gate=Linear(hidden, mlp, gen), up=Linear(hidden, mlp, gen), down=Linear(mlp, hidden, gen),
                cache=dq.KVCache.empty(pages, kv_heads, D, page_size, bits, device=device)))
        self.norm = torch.ones(hidden, dtype=torch.float16, device=device)
        self.head = Linear(hidden, vocab, gen)
        self.pool = dq.PagePool(pages, page_size)

    # ---- sequences
    def add(self, seq) -> None:
        self.pool.add(seq)

    def fork(self, seq, new) -> None:
        """`new` goes on from where `seq` is; full pages are shared."""
        self._copy(self.pool.fork(seq, new))

    def free(self, seq) -> None:
        self.pool.free(seq)

    def compact(self) -> None:
        self._copy(self.pool.compact())

    def _copy(self, pairs) -> None:
        if pairs:
            dq.copy_pages([layer["cache"] for layer in self.layers],
                          torch.tensor(pairs, dtype=torch.int32, device=self.device))

    # ---- one step
    def step(self, batch: list[tuple[object, list[int]]]) -> torch.Tensor:
        """Append each sequence's new tokens; logits float16 [tokens][vocab] of all of them.
        Raises MemoryError, changing nothing, if the pool has too few free pages."""
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=self.device)    # noqa: E731
        tokens, positions, slots, starts, lens = [], [], [], [0], []
        for seq, new in batch:
            at = self.pool.length(seq)
            try:
                slots += self.pool.extend(seq, len(new))
            except MemoryError:
                for (done, taken) in reversed(batch[:len(lens)]):
                    self.pool.truncate(done, self.pool.length(done) - len(taken))
                raise
            positions += range(at, at + len(new))
            tokens += new
            starts.append(len(tokens))
            lens.append(at + len(new))
        pages = [self.pool.pages(seq) for seq, _ in batch]
        width = max(map(len, pages))
        where = dict(block_table=ints([p + [0] * (width - len(p)) for p in pages]), kv_len=ints(lens),
                     q_start=ints(starts), max_q_len=max(len(new) for _, new in batch), max_kv_len=max(lens),
                     window=self.window)
        return self.forward(ints(tokens), ints(positions), ints(slots), where)

    def forward(self, tokens, positions, slots, where) -> torch.Tensor:
        T, H, Hk, D = tokens.shape[0], self.heads, self.kv_heads, self.dim
        workspace = dq.paged_attention_workspace(self.layers[0]["cache"], T, H, where["kv_len"].shape[0],
                                                 where["max_q_len"], where["max_kv_len"], self.device, self.window)
        x = self.embedding[tokens]
        delta = None                              # the previous block's output, added by the next norm
        for layer in self.layers:
            y = dq.rms_norm(x, layer["norms"][0], residual=delta, residual_out=None if delta is None else x)
            qkv = layer["qkv"](y).view(T, H + 2 * Hk, D)
            q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
            dq.rope_append(layer["cache"], q, k, v, positions, slots, self.table, q_out=q)
            y = dq.paged_attention(layer["cache"], q, workspace=workspace, **where)
            y = dq.rms_norm(layer["out"](y.view(T, H * D)), layer["norms"][1], residual=x, residual_out=x)
            delta = layer["down"](layer["gate"](y, activation=dq.ACT_SILU).mul_(layer["up"](y)))
        return self.head(dq.rms_norm(x, self.norm, residual=delta))


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("layers", 4), ("hidden", 4096), ("heads", 32), ("kv-heads", 8), ("mlp", 11008),
                        ("bits", 16), ("prompt", 1000), ("steps", 32), ("window", 0)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    d = Decoder(a.layers, a.hidden, a.heads, a.kv_heads, a.mlp, bits=a.bits, window=a.window,
                max_pos=a.prompt + a.steps + 1, pages=5 + 5 * (a.prompt + a.steps) // 64)
    prompt = torch.randint(0, 32000, (a.prompt,), generator=torch.Generator().manual_seed(1)).tolist()

    def timed(f):
        torch.cuda.synchronize()
        t = time.perf_counter()
        r = f()
        torch.cuda.synchronize()
        return r, (time.perf_counter() - t) * 1e3

    d.add("warm")
    d.step([("warm", prompt)])
    d.free("warm")
    d.add("a")
    logits, ms = timed(lambda: d.step([("a", prompt)]))
    print(f"prompt of {a.prompt} tokens, {a.layers} layers: {ms:.2f} ms")
    names = ["a", "b", "c", "d"]
    nxt = logits[-1].topk(4).indices.tolist()     # four branches, each with its own next token
    for name in names[1:]:
        d.fork("a", name)
    held = d.pool.num_pages - d.pool.free_pages
    print(f"four branches hold {held} pages; apart they would hold {4 * len(d.pool.pages('a'))}")

    def decode():
        tokens = nxt
        for _ in range(a.steps):
            tokens = d.step([(n, [t]) for n, t in zip(names, tokens)]).argmax(-1).tolist()
        return tokens

    _, ms = timed(decode)
    print(f"{a.steps} steps of four branches: {ms / a.steps:.3f} ms each")
    for name in names[:3]:
        d.free(name)
    d.compact()
    logits = d.step([("d", [nxt[3]])])
    print(f"one branch left, {d.pool.num_pages - d.pool.free_pages} pages in use, "
          f"logits finite: {bool(torch.isfinite(logits).all())}")


if __name__ == "__main__":
    main()
