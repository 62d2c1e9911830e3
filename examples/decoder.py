"""A decoder with quantized layers and a paged key/value cache, serving
sequences that come, share a prompt, branch and go: the library's calls in the
order in which a server makes them. Weights are random.

    python examples/decoder.py [--layers 4] [--hidden 4096] [--heads 32] [--kv-heads 8] [--bits 16]
                               [--window 0] [--sinks 0] [--head-norms 0] [--share 2]

prints the times of a prompt, of single-token steps over four branches of it,
the pages that the branches share, and how likely the prompt and the branches are.
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


# Decoder(share=): never, wherever sequences share a page, where they gain by it.
SHARE_NEVER, SHARE_ALWAYS, SHARE_GAINS = 0, 1, 2
# Branches gain from about so many on, behind so many tokens, with up to so many new
# ones each on average (us, shared and each by itself, float16: 8 single tokens behind
# 4096 27 and 29 with 64/8 heads, 20 and 28 with 32/8, 26 and 57 with 32/32; with 64/8
# 16 with 4 new ones 43 and 51, a prompt of 100 among 64 single tokens behind 16384 183
# and 683, but 16 with 16 new ones 77 and 78, 16 single ones behind 1024 27 and 20).
GAINS_SEQUENCES, GAINS_TOKENS, GAINS_NEW = 8, 4096, 4


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
    its new tokens: whole prompts, parts of them, drafts, single tokens.

    sinks: first tokens that a window leaves in sight; head_norms: the heads of q
    and k are normed before the rotation; share: whether neighbours in a batch that
    are branches of one sequence read the pages they share once for all of them
    (SHARE_NEVER, SHARE_ALWAYS or True, SHARE_GAINS)."""

    sinks, share = 0, SHARE_NEVER

    def __init__(self, layers: int = 4, hidden: int = 4096, heads: int = 32, kv_heads: int = 8, mlp: int = 11008,
                 vocab: int = 32000, pages: int = 256, page_size: int = 64, max_pos: int = 8192, bits: int = 16,
                 window: int = 0, seed: int = 0, device="cuda", sinks: int = 0, head_norms: bool = False,
                 share: int = SHARE_NEVER):
        gen = torch.Generator(device=device).manual_seed(seed)
        D = hidden // heads
        self.heads, self.kv_heads, self.dim, self.window, self.device = heads, kv_heads, D, window, torch.device(device)
        self.sinks, self.share = sinks, share
        self.embedding = torch.randn((vocab, hidden), generator=gen, device=device).half()
        self.table = dq.rope_table(max_pos, D, device=device)
        self.layers = []
        for _ in range(layers):
            norms = [(1 + 0.1 * torch.randn(hidden, generator=gen, device=device)).half() for _ in range(2)]
            self.layers.append(dict(
                norms=norms, qkv=Linear(hidden, (heads + 2 * kv_heads) * D, gen), out=Linear(hidden, hidden, gen),
                gate=Linear(hidden, mlp, gen), up=Linear(hidden, mlp, gen), down=Linear(mlp, hidden, gen),
                cache=dq.KVCache.empty(pages, kv_heads, D, page_size, bits, device=device)))
        for layer in self.layers:
            layer["head_norms"] = [(1 + 0.1 * torch.randn(D, generator=gen, device=device)).half() if head_norms else None
                                   for _ in range(2)]
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
        groups, shared = self._branches(batch)
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
        if any(shared):
            del where["window"]                   # there is none, and sinks are seen without one
            where.update(shared_start=ints(groups), shared_len=ints(shared), max_shared_len=max(shared))
        elif self.sinks:
            where["sinks"] = self.sinks
        return self.forward(ints(tokens), ints(positions), ints(slots), where)

    def _branches(self, batch) -> tuple[list[int], list[int]]:
        """Neighbours that share pages: where each group starts, and what it shares (a window sees too
        little of it)."""
        seqs = [seq for seq, _ in batch]
        groups, shared = [0], []
        while self.share and self.window == 0 and groups[-1] < len(seqs):
            at, n, tokens = groups[-1], 1, 0
            while at + n < len(seqs):
                more = self.pool.shared_tokens(seqs[at:at + n + 1])
                if more < max(self.pool.page_size, tokens // 2):
                    break
                n, tokens = n + 1, more
            gains = (n >= GAINS_SEQUENCES and tokens >= GAINS_TOKENS
                     and sum(len(new) for _, new in batch[at:at + n]) <= GAINS_NEW * n)
            groups.append(at + n)
            shared.append(tokens if gains or self.share != SHARE_GAINS else 0)
        return groups, shared

    def forward(self, tokens, positions, slots, where) -> torch.Tensor:
        T, H, Hk, D = tokens.shape[0], self.heads, self.kv_heads, self.dim
        sizes = self.layers[0]["cache"], T, H, where["kv_len"].shape[0], where["max_q_len"], where["max_kv_len"]
        if "shared_len" in where:
            attention = dq.paged_attention_shared
            workspace = dq.paged_attention_shared_workspace(*sizes, where["shared_len"].shape[0],
                                                            where["max_shared_len"], self.device)
        else:
            attention = dq.paged_attention
            workspace = dq.paged_attention_workspace(*sizes, self.device, self.window, where.get("sinks", 0))
        x = self.embedding[tokens]
        delta = None                              # the previous block's output, added by the next norm
        for layer in self.layers:
            y = dq.rms_norm(x, layer["norms"][0], residual=delta, residual_out=None if delta is None else x)
            qkv = layer["qkv"](y).view(T, H + 2 * Hk, D)
            q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
            q_norm, k_norm = layer["head_norms"]
            dq.rope_append(layer["cache"], q, k, v, positions, slots, self.table, q_out=q, q_norm=q_norm,
                           k_norm=k_norm)
            y = attention(layer["cache"], q, workspace=workspace, **where)
            y = dq.rms_norm(layer["out"](y.view(T, H * D)), layer["norms"][1], residual=x, residual_out=x)
            delta = layer["down"](layer["gate"](y, activation=dq.ACT_SILU).mul_(layer["up"](y)))
        return self.head(dq.rms_norm(x, self.norm, residual=delta))


def arguments(args=None) -> argparse.Namespace:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("layers", 4), ("hidden", 4096), ("heads", 32), ("kv-heads", 8), ("mlp", 11008),
                        ("bits", 16), ("prompt", 1000), ("steps", 32), ("window", 0), ("sinks", 0), ("head-norms", 0),
                        ("share", SHARE_GAINS)):
        p.add_argument("--" + name, type=int, default=value)
    return p.parse_args(args)


def main() -> None:
    a = arguments()
    d = Decoder(a.layers, a.hidden, a.heads, a.kv_heads, a.mlp, bits=a.bits, window=a.window,
                sinks=a.sinks, head_norms=bool(a.head_norms), share=a.share,
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
    said = dq.token_logprobs(logits[:-1], torch.tensor(prompt[1:], dtype=torch.int32, device=d.device))
    print(f"its tokens' mean log probability: {said.logprob.mean().item():.3f}, entropy {said.entropy.mean().item():.3f}")
    names = ["a", "b", "c", "d"]
    first = dq.token_logprobs(logits[-1:], top=4, entropy=False)     # four branches, each with its own next token
    nxt, likely = first.top_id[0].tolist(), first.top_logprob[0].clone()
    for name in names[1:]:
        d.fork("a", name)
    held = d.pool.num_pages - d.pool.free_pages
    print(f"four branches hold {held} pages; apart they would hold {4 * len(d.pool.pages('a'))}")

    def decode():
        tokens = nxt
        for _ in range(a.steps):
            best = dq.token_logprobs(d.step([(n, [t]) for n, t in zip(names, tokens)]), top=1, entropy=False)
            likely.add_(best.top_logprob[:, 0])
            tokens = best.top_id[:, 0].tolist()
        return tokens

    _, ms = timed(decode)
    print(f"{a.steps} steps of four branches: {ms / a.steps:.3f} ms each")
    print("the branches' log probabilities: " + ", ".join(f"{x:.2f}" for x in likely.tolist()))
    for name in names[:3]:
        d.free(name)
    d.compact()
    logits = d.step([("d", [nxt[3]])])
    print(f"one branch left, {d.pool.num_pages - d.pool.free_pages} pages in use, "
          f"logits finite: {bool(torch.isfinite(logits).all())}")


if __name__ == "__main__":
    main()
