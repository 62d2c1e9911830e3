"""Operators of a decoder's serving path that stand around its paged cache, as
cases to measure: norms of queries and keys with the rotary append, attention
with a sliding window and first tokens that stay visible (sinks), attention for
a batch that shares a long prefix, and log probabilities of given tokens with
entropy and top alternatives. `own` selects between the elementary torch form
(False) and this package's kernels (True).

Head counts: 32 heads of 128 (hidden 4096), 64 query and 8 key/value heads
(hidden 8192); 64- and 256-wide heads and the other counts are generic.
Vocabulary sizes: 32000, and generic ones.

Cache pools: K and V are [pages][kv_heads][page][dim] float16, or for 8, 6 and
4 bits codes int32 [pages][kv_heads][page][dim * bits / 32] (a little-endian
bit stream per row) with float16 scales [pages][kv_heads][page][dim / group]; a
value is scale * (code - 2^(bits-1)) rounded to float16.
"""

from __future__ import annotations

import math

import torch

own = False

ROPE_BASE = 10000.0
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One user's token on the grouped-head model: the smallest call, where
        # latency counts.
        dict(name="norm-rope-1-h64kv8", op="rope", tokens=1, q_heads=64, kv_heads=8, dim=128, rot=128, layout="half",
             weights="one", page=256, bits=16, group=128, max_pos=8192),
        # A few hundred tokens of several sequences (a chunk of a prompt and
        # single tokens) into a 4-bit cache: wide heads, a quarter of them
        # rotated, a weight for every head.
        dict(name="norm-rope-333-q4-h24kv8-d256", op="rope", tokens=333, q_heads=24, kv_heads=8, dim=256, rot=64,
             layout="interleaved", weights="heads", page=16, bits=4, group=32, max_pos=32768),
        # A long prompt's rotary step into an 8-bit cache.
        dict(name="norm-rope-8191-q8-h64kv8", op="rope", tokens=8191, q_heads=64, kv_heads=8, dim=128, rot=128,
             layout="half", weights="one", page=64, bits=8, group=64, max_pos=131072),
        # One stream that has run for long behind a window, a token at a time.
        dict(name="sinks-decode-1x30001-w1024", op="sinks", q_heads=32, kv_heads=32, dim=128, page=256, bits=16,
             group=128, q_lens="1", kv_lens="30001", window=1024, sinks=4),
        # A serving batch of streams of all ages over an 8-bit cache, some
        # shorter than the window, drafts of up to 4 tokens among them.
        dict(name="sinks-decode-40xragged-q8-h64kv8", op="sinks", q_heads=64, kv_heads=8, dim=128, page=64, bits=8,
             group=128, q_lens="1x36,4x4",
             kv_lens="65000,1,40,4100,9001,33333,2047,12000,5000x3,777,64,20000,4096,4097,31,8191,10001x10,300,1500,2500,"
                     "3500,4500,5500,6500,7500,30000,6000,7000,9500", window=4096, sinks=64),
        # A prompt of 6000 tokens through a layer with a window.
        dict(name="sinks-prompt-6000-w1024-h32kv8", op="sinks", q_heads=32, kv_heads=8, dim=128, page=256, bits=16,
             group=128, q_lens="6000", kv_lens="6000", window=1024, sinks=4),
        # Eight branches of one conversation of 2000 tokens on the 32-head
        # model, each some way on: few rows, the smallest shared call.
        dict(name="shared-decode-8x2000-h32", op="shared", q_heads=32, kv_heads=32, dim=128, page=16, bits=16, group=128,
             groups="8", shared="2000", q_lens="1x8", tails="1,17,300,64,129,5,250,33"),
        # A serving batch behind one system prompt with documents in it.
        dict(name="shared-decode-32x16k-h64kv8", op="shared", q_heads=64, kv_heads=8, dim=128, page=256, bits=16,
             group=128, groups="32", shared="16384", q_lens="1x32",
             tails="900,1,300,44,512,700,128,257,60,5,1000,333,80,650,17,220,410,99,31,800,3,150,270,600,720,12,480,"
                   "555,350,64,201,96"),
        # Three prompts of many users, with drafts of 4 tokens to verify,
        # over an 8-bit cache.
        dict(name="shared-drafts-3groups-q8-h64kv8", op="shared", q_heads=64, kv_heads=8, dim=128, page=64, bits=8,
             group=64, groups="20,9,1", shared="8192,4096,640", q_lens="4x30",
             tails="40,300,8,77,150,4,222,63,500,35,91,18,260,410,5,120,33,64,87,199,350,24,600,71,5,140,96,31,7,900"),
        # Six questions about one document arrive at once: prompts behind the
        # shared prefix, the largest call.
        dict(name="shared-prompts-6x8192-h64kv8", op="shared", q_heads=64, kv_heads=8, dim=128, page=256, bits=16,
             group=128, groups="6", shared="8192", q_lens="333,512,100,257,700,41", tails="333,512,100,257,700,41"),
        # The next token's distribution for one user, after a sampler's
        # penalties and masks in 32 bits, over a large vocabulary.
        dict(name="logprob-1x131072-f32-top20", op="logprob", tokens=1, vocab=131072, top=20, dtype="f32", masked=True),
        # A prompt's tokens scored.
        dict(name="logprob-2047x32000-top5", op="logprob", tokens=2047, vocab=32000, top=5, dtype="f16", masked=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = ((32, 32), (64, 8), (32, 8), (32, 4), (24, 8), (20, 4), (16, 1))


def _draw_cache(rng):
    bits = rng.choice((16, 16, 8, 6, 4))
    dim = rng.choice((64, 128, 128, 128, 256))
    c = dict(bits=bits, dim=dim, group=rng.choice([g for g in (32, 64, 128) if dim % g == 0]),
             page=rng.choice((16, 32, 64, 128, 256)))
    c["q_heads"], c["kv_heads"] = rng.choice(_HEADS)
    return c


def draw(rng):
    op = rng.choice(("rope", "sinks", "sinks", "shared", "shared", "logprob"))
    if op == "logprob":
        vocab = rng.choice((32000, 32001, 65536, _log_int(rng, 500, 262144)))
        return dict(op=op, tokens=_log_int(rng, 1, max(1, 2047 * 32000 // vocab)), vocab=vocab,
                    top=rng.choice((0, 1, 5, 20, 64)), dtype=rng.choice(("f16", "f16", "f32")),
                    masked=rng.random() < 0.5)
    c = dict(op=op, **_draw_cache(rng))
    if op == "rope":
        c["tokens"] = _log_int(rng, 1, 8191 * 64 * 128 // (c["q_heads"] * c["dim"]) // 2)
        c["rot"] = rng.choice((c["dim"], c["dim"], c["dim"] // 2, c["dim"] // 4))
        c["layout"] = rng.choice(("half", "interleaved"))
        c["weights"] = rng.choice(("one", "one", "heads"))
        c["max_pos"] = max(c["tokens"], _log_int(rng, 64, 131072))
        return c
    chunk = rng.random() < 0.35
    if op == "sinks":
        c["window"], c["sinks"] = _log_int(rng, 16, 8192), rng.choice((1, 4, 64, _log_int(rng, 1, 300)))
        if chunk:
            n = rng.choice((1, 1, 3))
            q = [_log_int(rng, 16, 5000 // n) for _ in range(n)]
            while 4.0 * c["q_heads"] * sum(x * (x + c["window"]) for x in q) > 2e9:
                q = [max(1, x * 3 // 4) for x in q]
        else:
            q = [rng.choice((1, 1, 1, 2, 4, 7))] * _log_int(rng, 1, 48)
        kv = [x + _log_int(rng, 1, 40000) - 1 for x in q]
        while sum(kv) * c["kv_heads"] * c["dim"] * 4 > 4e9:
            kv = [max(x, y // 2) for x, y in zip(q, kv)]
        c["q_lens"], c["kv_lens"] = ",".join(map(str, q)), ",".join(map(str, kv))
        return c
    sizes = [_log_int(rng, 1, 32) for _ in range(rng.choice((1, 1, 2, 4)))]
    n = sum(sizes)
    shared = [c["page"] * max(1, _log_int(rng, 1, 16384) // c["page"]) for _ in sizes]
    if chunk:
        q = [_log_int(rng, 2, max(2, 1500 // n)) for _ in range(n)]
        tails = list(q)
    else:
        q = [rng.choice((1, 1, 1, 2, 4, 7))] * n
        tails = [x + _log_int(rng, 1, 1000) - 1 for x in q]
    while len(sizes) * sum(q) * c["q_heads"] * max(shared) > 1e9:
        shared = [max(c["page"], s // 2 // c["page"] * c["page"]) for s in shared]
    c["groups"], c["shared"] = ",".join(map(str, sizes)), ",".join(map(str, shared))
    c["q_lens"], c["tails"] = ",".join(map(str, q)), ",".join(map(str, tails))
    return c


# ---------------------------------------------------------------- inputs

def _lens(text):
    out = []
    for part in text.split(","):
        a, _, n = part.partition("x")
        out += [int(a)] * (int(n) if n else 1)
    return out


def _spread(gen, shape):
    """Key/value-like rows: N(0, 1) with a magnitude per channel (a few channels several times larger)."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    return x.mul_(torch.exp(0.4 * torch.randn(shape[-1], generator=gen, device="cuda")).to(torch.float16))


# codes that fill whole bytes together, and the bytes
_UNIT = {8: (1, 1), 6: (4, 3), 4: (2, 1)}


def _pack(q, bits):
    """Codes int32 [..., D] -> words int32 [..., D * bits / 32]."""
    n, nb = _UNIT[bits]
    unit = (q.unflatten(-1, (-1, n)) << (bits * torch.arange(n, device=q.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    b = (unit.unsqueeze(-1) >> (8 * torch.arange(nb, device=q.device, dtype=torch.int32))) & 255
    return b.to(torch.uint8).flatten(-2).contiguous().view(torch.int32)


def _encode(x, bits, group):
    """float16 [..., D] -> (words, float16 scales [..., D / group])."""
    half = 1 << (bits - 1)
    xf = x.float().unflatten(-1, (-1, group))
    s = (xf.abs().amax(-1) / float(half - 1)).to(torch.float16)
    sf = s.float().unsqueeze(-1)
    r = torch.where(sf > 0, torch.round(xf / torch.where(sf > 0, sf, torch.ones_like(sf))), torch.zeros_like(xf))
    return _pack((r.clamp(-half, half - 1) + half).to(torch.int32).flatten(-2), bits), s


def _values(words, scales, bits):
    """float16 values that codes and scales stand for."""
    n, nb = _UNIT[bits]
    b = words.contiguous().view(torch.uint8).unflatten(-1, (-1, nb)).to(torch.int32)
    unit = (b << (8 * torch.arange(nb, device=b.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    q = (unit.unsqueeze(-1) >> (bits * torch.arange(n, device=b.device, dtype=torch.int32))) & ((1 << bits) - 1)
    q = (q.flatten(-2) - (1 << (bits - 1))).float().unflatten(-1, (scales.shape[-1], -1))
    return (q * scales.float().unsqueeze(-1)).flatten(-2).to(torch.float16)


def _pools(gen, case, pages):
    """Pools of rows as _spread makes them, encoded for 8, 6 and 4 bits."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    p = {}
    for name in ("k", "v"):
        x = _spread(gen, shape)
        if case["bits"] == 16:
            p[name] = x
            continue
        parts = [_encode(part, case["bits"], case["group"]) for part in x.split(max(1, (1 << 25) // x[0].numel()))]
        p[name], p[name + "_scales"] = (torch.cat(t) for t in zip(*parts))
    return p


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "logprob":
        _prepare_logprob(st, case, gen)
    elif case["op"] == "rope":
        _prepare_rope(st, case, gen)
    else:
        _prepare_attention(st, case, gen)
    return st


def _prepare_logprob(st, case, gen):
    T, V = case["tokens"], case["vocab"]
    # Logits as heads give them: N(0, 3), and some confident rows.
    x = torch.randn((T, V), generator=gen, device="cuda") * 3
    tokens = torch.randint(0, V, (T,), generator=gen, device="cuda")
    sure = torch.rand(T, generator=gen, device="cuda") < 0.4
    x[torch.arange(T, device="cuda"), tokens] += torch.where(sure, 14.0, 0.0)
    if case["masked"]:            # a grammar leaves half of the vocabulary
        hidden = torch.rand((T, V), generator=gen, device="cuda") < 0.5
        hidden[torch.arange(T, device="cuda"), tokens] = False
        x.masked_fill_(hidden, -math.inf)
    st["logits"] = x.to(torch.float16) if case["dtype"] == "f16" else x
    st["tokens"] = tokens.to(torch.int32)


def _prepare_rope(st, case, gen):
    T, P, D = case["tokens"], case["page"], case["dim"]
    pages = -(-T // P) + 2
    st["pools"] = _pools(gen, case, pages)
    for name, heads in (("q", case["q_heads"]), ("k", case["kv_heads"]), ("v", case["kv_heads"])):
        st[name] = _spread(gen, (T, heads, D))
    for name, heads in (("q_norm", case["q_heads"]), ("k_norm", case["kv_heads"])):
        w = 1 + 0.3 * torch.randn((heads, D) if case["weights"] == "heads" else (D,), generator=gen, device="cuda")
        st[name] = w.to(torch.float16)
    first = int(torch.randint(0, case["max_pos"] - T + 1, (1,), generator=gen, device="cuda"))
    st["positions"] = torch.arange(first, first + T, device="cuda", dtype=torch.int32)
    order = torch.randperm(pages, generator=gen, device="cuda")
    i = torch.arange(T, device="cuda")
    st["slots"] = (order[i // P] * P + i % P).to(torch.int32)
    half = case["rot"] // 2
    inv = ROPE_BASE ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    ang = torch.arange(case["max_pos"], dtype=torch.float64, device="cuda").unsqueeze(1) * inv
    st["table"] = torch.stack((torch.cos(ang), torch.sin(ang)), -1).float()
    st["q_out"] = torch.empty_like(st["q"])
    if own:
        st["cache"] = _cache(case, st["pools"])


def _prepare_attention(st, case, gen):
    P = case["page"]
    ql = _lens(case["q_lens"])
    if case["op"] == "sinks":
        kl, head, sizes, shared = _lens(case["kv_lens"]), [0] * len(ql), [len(ql)], [0]
    else:
        sizes, shared, tails = _lens(case["groups"]), _lens(case["shared"]), _lens(case["tails"])
        head = [s // P for s, n in zip(shared, sizes) for _ in range(n)]      # shared pages of each sequence
        kl = [h * P + t for h, t in zip(head, tails)]
    own_pages = [-(-l // P) - h for l, h in zip(kl, head)]
    common = [s // P for s in shared]
    pages = sum(own_pages) + sum(common) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(kl), max(h + n for h, n in zip(head, own_pages))), -1, dtype=torch.int32, device="cuda")
    at = b = 0
    for n, size in zip(common, sizes):
        for i in range(b, b + size):
            table[i, :n] = order[at:at + n]
        at, b = at + n, b + size
    for b, (h, n) in enumerate(zip(head, own_pages)):
        table[b, h:h + n] = order[at:at + n]
        at += n
    st["pools"] = _pools(gen, case, pages)
    st["q"] = torch.randn((sum(ql), case["q_heads"], case["dim"]), generator=gen, device="cuda", dtype=torch.float16)
    st["table"], st["kv_len"], st["q_start"] = table, _ints(kl), _ints(_starts(ql))
    st["shared_start"], st["shared_len"] = _ints(_starts(sizes)), _ints([n * P for n in common])
    st["q_lens"], st["kv_lens"], st["sizes"], st["shared_lens"] = ql, kl, sizes, [n * P for n in common]
    if own:
        import dequant_matmul_gptq_amd as dq
        st["cache"], st["out"] = _cache(case, st["pools"]), torch.empty_like(st["q"])
        sizes = (st["cache"], sum(ql), case["q_heads"], len(ql), max(ql), max(kl))
        if case["op"] == "sinks":
            st["workspace"] = dq.paged_attention_workspace(*sizes, "cuda", window=case["window"], sinks=case["sinks"])
        else:
            st["workspace"] = dq.paged_attention_shared_workspace(*sizes, len(common), max(st["shared_lens"]), "cuda")


def _cache(case, pools):
    import dequant_matmul_gptq_amd as dq
    return dq.KVCache(pools["k"], pools["v"], pools.get("k_scales"), pools.get("v_scales"), head_dim=case["dim"])


# ---------------------------------------------------------------- one pass

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import dequant_matmul_gptq_amd as dq
    case = st["case"]
    if case["op"] == "logprob":
        r = dq.token_logprobs(st["logits"], st["tokens"], top=case["top"])
        return (r.logprob, r.entropy) + ((r.top_logprob, r.top_id) if case["top"] else ())
    if case["op"] == "rope":
        layout = dq.ROPE_HALF if case["layout"] == "half" else dq.ROPE_INTERLEAVED
        dq.rope_append(st["cache"], st["q"], st["k"], st["v"], st["positions"], st["slots"], st["table"],
                       layout=layout, q_out=st["q_out"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS)
        p = st["pools"]
        if case["bits"] == 16:
            return st["q_out"], p["k"], p["v"]
        return (st["q_out"],) + tuple(dq.kv_dequant(p[n], p[n + "_scales"], case["dim"], case["bits"], case["group"])
                                      for n in ("k", "v"))
    bounds = dict(max_q_len=max(st["q_lens"]), max_kv_len=max(st["kv_lens"]), out=st["out"], workspace=st["workspace"])
    if case["op"] == "sinks":
        return dq.paged_attention(st["cache"], st["q"], st["table"], st["kv_len"], st["q_start"],
                                  window=case["window"], sinks=case["sinks"], **bounds)
    return dq.paged_attention_shared(st["cache"], st["q"], st["table"], st["kv_len"], st["shared_len"],
                                     st["shared_start"], st["q_start"], max_shared_len=max(st["shared_lens"]), **bounds)


def _run_plain(st):
    return {"logprob": _plain_logprob, "rope": _plain_rope, "sinks": _plain_sinks, "shared": _plain_shared}[st["case"]["op"]](st)


def _plain_logprob(st):
    x, k = st["logits"].float(), st["case"]["top"]
    V = x.shape[1]
    z = x - x.amax(-1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(-1)
    lse = torch.log(total)
    logprob = z.gather(1, st["tokens"].long().unsqueeze(1)).squeeze(1) - lse
    entropy = lse - torch.where(e > 0, e * z, torch.zeros_like(z)).sum(-1) / total
    if not k:
        return logprob, entropy
    # Distinct keys: the value's order first, then the lower index.
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits) * 2 ** 31 + (V - 1 - torch.arange(V, device=x.device))
    ids = V - 1 - (torch.topk(key, k, dim=-1).values & (2 ** 31 - 1))
    return logprob, entropy, z.gather(1, ids) - lse.unsqueeze(1), ids.to(torch.int32)


def _normed(x, w):
    x = x.float()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _plain_rope(st):
    case, p = st["case"], st["pools"]
    r = case["rot"]
    a, b = (slice(0, r // 2), slice(r // 2, r)) if case["layout"] == "half" else (slice(0, r, 2), slice(1, r, 2))
    cs = st["table"][st["positions"].long()].unsqueeze(1)

    def turned(x):
        y = x.clone()
        y[..., a] = x[..., a] * cs[..., 0] - x[..., b] * cs[..., 1]
        y[..., b] = x[..., b] * cs[..., 0] + x[..., a] * cs[..., 1]
        return y.to(torch.float16)

    st["q_out"].copy_(turned(_normed(st["q"], st["q_norm"])))
    pg, off = st["slots"].long() // case["page"], st["slots"].long() % case["page"]
    k = turned(_normed(st["k"], st["k_norm"]))
    if case["bits"] == 16:
        p["k"][pg, :, off], p["v"][pg, :, off] = k, st["v"]
        return st["q_out"], p["k"], p["v"]
    p["k"][pg, :, off], p["k_scales"][pg, :, off] = _encode(k, case["bits"], case["group"])
    p["v"][pg, :, off], p["v_scales"][pg, :, off] = _encode(st["v"], case["bits"], case["group"])
    return st["q_out"], _values(p["k"], p["k_scales"], case["bits"]), _values(p["v"], p["v_scales"], case["bits"])


def _cached(st, name, table, t):
    """float32 [sequences][kv_heads][tokens][dim]: tokens t [sequences][tokens] behind the rows of the block table."""
    p, case = st["pools"], st["case"]
    page = table.long().gather(1, t // case["page"]).clamp(min=0)
    x = p[name][page, :, t % case["page"]]
    if case["bits"] != 16:
        x = _values(x, p[name + "_scales"][page, :, t % case["page"]], case["bits"])
    return x.transpose(1, 2).float()


def _padded(st, start, count, width):
    """(float32 [batches][kv_heads][heads of a group * width][dim], places int64 [rows of q]): the rows of q from
    start on, in batches of `width`, and where each of them went."""
    case, q = st["case"], st["q"]
    Hk, D = case["kv_heads"], case["dim"]
    rows = (start.unsqueeze(1) + torch.arange(width, device="cuda")).clamp(max=q.shape[0] - 1)
    x = q[rows].float().view(len(start), width, Hk, -1, D).permute(0, 2, 3, 1, 4)
    r = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(start + count, r, right=True)
    return x.reshape(len(start), Hk, -1, D), b * width + r - start[b]


def _scores(q, k, hidden, group):
    """exp(score - max), max and sum of each row; hidden [batches][rows or 1][tokens]."""
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(q.shape[-1]))
    s = s.view(*s.shape[:2], group, -1, s.shape[-1]).masked_fill_(hidden[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s = s.sub_(m).exp_()
    return s.flatten(2, 3), m, s.sum(-1, keepdim=True)


def _by_token(x, places, width):
    """[batches][kv_heads][heads of a group][width][.] -> [tokens][q_heads][.]."""
    return x.permute(0, 3, 1, 2, 4).flatten(2, 3).flatten(0, 1)[places]


def _plain_sinks(st):
    case = st["case"]
    G, w, S = case["q_heads"] // case["kv_heads"], case["window"], case["sinks"]
    ql, kl = st["q_lens"], st["kv_lens"]
    L, start = st["kv_len"].long(), st["q_start"].long()
    n = start[1:] - start[:-1]
    low = (L - n - w + 1).clamp(min=0).unsqueeze(1)
    # The first tokens, and from the first one in a window on.
    first = torch.arange(S, device="cuda").expand(len(ql), S)
    rest = low + torch.arange(max(l - max(0, l - x - w + 1) for x, l in zip(ql, kl)), device="cuda")
    t = torch.cat((torch.where(first < low, first, 1 << 30), rest), 1)
    q, places = _padded(st, start[:-1], n, max(ql))
    pos = (L - n).unsqueeze(1) + torch.arange(max(ql), device="cuda")
    t, pos = t.unsqueeze(1), pos.unsqueeze(2)
    hidden = (t > pos) | ((t <= pos - w) & (t >= S)) | (t >= L[:, None, None])
    at = torch.minimum(t.squeeze(1), (L - 1).unsqueeze(1)).clamp(min=0)
    e, _, total = _scores(q, _cached(st, "k", st["table"], at), hidden, G)
    o = torch.matmul(e, _cached(st, "v", st["table"], at)).view(*total.shape[:-1], -1) / total
    return _by_token(o, places, max(ql)).to(torch.float16)


def _plain_shared(st):
    case = st["case"]
    G = case["q_heads"] // case["kv_heads"]
    ql, L, start = st["q_lens"], st["kv_len"].long(), st["q_start"].long()
    n = start[1:] - start[:-1]
    first, S = st["shared_start"].long(), st["shared_len"].long()
    size = first[1:] - first[:-1]
    # The shared tokens, once for all rows of a group.
    rows = start[first[1:]] - start[first[:-1]]
    at = _starts(st["sizes"])
    width = max(sum(ql[a:b]) for a, b in zip(at, at[1:]))
    t = torch.arange(max(st["shared_lens"]), device="cuda").expand(len(S), -1)
    q, places = _padded(st, start[first[:-1]], rows, width)
    hidden = (t >= S.unsqueeze(1)).unsqueeze(1)
    inside = torch.minimum(t, (S - 1).unsqueeze(1)).clamp(min=0)
    table = st["table"][first[:-1]]
    e, m, l = _scores(q, _cached(st, "k", table, inside), hidden, G)
    o = torch.matmul(e, _cached(st, "v", table, inside)).view(*l.shape[:-1], -1)
    o, m, l = (_by_token(x, places, width) for x in (o, m, l))
    # Each sequence's own tokens.
    low = torch.repeat_interleave(S, size, output_size=len(ql)).unsqueeze(1)
    own_len = max(l - s for l, s in zip(st["kv_lens"], [s for s, c in zip(st["shared_lens"], st["sizes"]) for _ in range(c)]))
    t = low + torch.arange(own_len, device="cuda")
    q, places = _padded(st, start[:-1], n, max(ql))
    pos = (L - n).unsqueeze(1) + torch.arange(max(ql), device="cuda")
    hidden = t.unsqueeze(1) > pos.unsqueeze(2)
    inside = torch.minimum(t, (L - 1).unsqueeze(1))
    e, m2, l2 = _scores(q, _cached(st, "k", st["table"], inside), hidden, G)
    o2 = torch.matmul(e, _cached(st, "v", st["table"], inside)).view(*l2.shape[:-1], -1)
    o2, m2, l2 = (_by_token(x, places, max(ql)) for x in (o2, m2, l2))
    top = torch.maximum(m, m2)
    f, f2 = torch.exp(m - top), torch.exp(m2 - top)
    return ((f * o + f2 * o2) / (f * l + f2 * l2)).to(torch.float16)


# ---------------------------------------------------------------- bytes and operations

def _row_bytes(case):
    if case["bits"] == 16:
        return 2 * case["dim"]
    return case["dim"] * case["bits"] // 8 + 2 * case["dim"] // case["group"]


def work(case):
    op = case["op"]
    if op == "logprob":
        n = case["tokens"] * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "f16" else 4) + case["tokens"] * (12 + 8 * case["top"]), "flops": 5 * n}
    D, Hq, Hk = case["dim"], case["q_heads"], case["kv_heads"]
    if op == "rope":
        T = case["tokens"]
        b = T * (2 * Hq * D * 2 + 2 * Hk * D * 2 + 4 * case["rot"] + 8) + T * Hk * 2 * _row_bytes(case)
        if case["bits"] != 16:                     # the pools come back as the values they stand for
            b += (-(-T // case["page"]) + 2) * case["page"] * Hk * 2 * (_row_bytes(case) + 2 * D)
        return {"bytes": b, "flops": T * (Hq + Hk) * (4 * D + 3 * case["rot"])}
    ql = _lens(case["q_lens"])
    rows = pairs = 0
    if op == "sinks":
        w, S = case["window"], case["sinks"]
        for n, L in zip(ql, _lens(case["kv_lens"])):
            low = max(0, L - n - w + 1)
            rows += L - low + min(low, S)
            for p in range(L - n, L):
                lo = max(0, p - w + 1)
                pairs += p + 1 - lo + min(lo, S)
    else:
        sizes, tails = _lens(case["groups"]), _lens(case["tails"])
        shared = [s // case["page"] * case["page"] for s in _lens(case["shared"])]
        at = _starts(sizes)
        for s, a, b in zip(shared, at, at[1:]):
            rows += s
            pairs += s * sum(ql[a:b])
        for n, t in zip(ql, tails):
            rows += t
            pairs += n * (t - n) + n * (n + 1) // 2
    return {"bytes": rows * Hk * 2 * _row_bytes(case) + 2 * sum(ql) * Hq * D * 2, "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprob":
        return _exact_logprob(st)
    if case["op"] == "rope":
        return _exact_rope(st)
    return _exact_attention(st)


def _exact_logprob(st):
    parts = []
    for x, token in zip(st["logits"].split(256), st["tokens"].long().split(256)):
        x = x.double()
        lp = x - torch.logsumexp(x, 1, keepdim=True)
        h = torch.special.entr(torch.exp(lp)).sum(1)
        row = [lp[torch.arange(len(x), device="cuda"), token], h]
        if st["case"]["top"]:
            ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :st["case"]["top"]]
            row += [torch.take_along_dim(lp, ids, 1), ids.to(torch.int32)]
        parts.append(row)
    return tuple(torch.cat(p) for p in zip(*parts))


def _stored(words, scales, case):
    """float64: the values of a pool's rows."""
    if case["bits"] == 16:
        return words.double()
    bits, D = case["bits"], case["dim"]
    w = words.long() & 0xFFFFFFFF
    i = torch.arange(D, device="cuda") * bits
    nxt = w[..., torch.clamp(i // 32 + 1, max=w.shape[-1] - 1)] << (32 - i % 32)
    q = w[..., i // 32] >> (i % 32)
    q = (torch.where(i % 32 + bits > 32, q | nxt, q) & ((1 << bits) - 1)).double() - 2.0 ** (bits - 1)
    return (q * scales.double().repeat_interleave(case["group"], -1)).to(torch.float16).double()


def _exact_rope(st):
    case, p = st["case"], st["pools"]
    T, P, r, D = case["tokens"], case["page"], case["rot"], case["dim"]
    cs = st["table"].double()[st["positions"].long()]
    z = torch.complex(cs[..., 0], cs[..., 1]).unsqueeze(1)
    done = {}
    for name in ("q", "k"):
        x = st[name].double()
        x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / D + EPS) * st[name + "_norm"].double()
        if case["layout"] == "half":
            u = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * z
            turned = torch.cat((u.real, u.imag), -1)
        else:
            u = torch.view_as_complex(x[..., :r].reshape(T, -1, r // 2, 2).contiguous()) * z
            turned = torch.view_as_real(u).reshape(T, -1, r)
        done[name] = torch.cat((turned, x[..., r:]), -1)
    out = [done["q"]]
    slot = st["slots"].long()
    for name, x in (("k", done["k"]), ("v", st["v"].double())):
        if case["bits"] != 16:
            half = 1 << (case["bits"] - 1)
            x = x.to(torch.float16).double().reshape(T, -1, D // case["group"], case["group"])
            s = (x.abs().amax(-1, keepdim=True) / (half - 1)).to(torch.float16).double()
            q = torch.where(s > 0, torch.round(x / s.clamp(min=1e-30)), torch.zeros_like(x)).clamp(-half, half - 1)
            x = (q * s).to(torch.float16).double().reshape(T, -1, D)
        pool = _stored(p[name], p.get(name + "_scales"), case)
        pool[slot // P, :, slot % P] = x
        out.append(pool)
    return tuple(out)


def _exact_attention(st):
    case, p = st["case"], st["pools"]
    Hq, Hk, D, P = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    w, S = case.get("window", 0), case.get("sinks", 0)
    res = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, L) in enumerate(zip(st["q_lens"], st["kv_lens"])):
        t = torch.arange(L, device="cuda")
        if w > 0:
            t = t[(t < S) | (t > L - n - w)]
        page = st["table"][b].long()[t // P]
        for c in range(Hk):
            k, v = (_stored(p[x][page, c, t % P], p[x + "_scales"][page, c, t % P] if case["bits"] != 16 else None, case)
                    for x in ("k", "v"))
            heads = slice(c * (Hq // Hk), (c + 1) * (Hq // Hk))
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                pos = torch.arange(L - n + i, L - n + i + m, device="cuda")
                z = st["q"][at + i:at + i + m, heads].double().transpose(0, 1) @ k.T / math.sqrt(D)
                see = t[None, :] <= pos[:, None]
                if w > 0:
                    see &= (t[None, :] < S) | (pos[:, None] - t[None, :] < w)
                z = z.masked_fill(~see, -math.inf)
                res[at + i:at + i + m, heads] = (torch.softmax(z, -1) @ v).transpose(0, 1)
        at += n
    return res
