"""The attention-side operators of a decoder layer, as cases to measure.

Each case is one call of an operator that stands between the quantized linear
layers of a Llama-shaped decoder: attention over a paged key/value cache,
rotary positions with the append to that cache, page copies, and the
root-mean-square norm with the residual's addition. `own` selects between the
elementary torch form (False) and this package's kernels (True).

Head counts: 32 heads of 128 (hidden 4096), 40 heads (hidden 5120), 64 query
and 8 key/value heads (hidden 8192); 64-wide heads are generic.

Cache pools: K and V are [pages][kv_heads][page_size][head_dim] float16, or
for 8, 6 and 4 bits codes int32 [pages][kv_heads][page_size][head_dim * bits /
32] (a little-endian bit stream per row) with float16 scales
[pages][kv_heads][page_size][head_dim / group]; a value is scale * (code -
2^(bits-1)) rounded to float16.
"""

from __future__ import annotations

import math

import torch

own = False

ROPE_BASE = 10000.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One user generating token by token on the 32-head model, about a
        # thousand tokens in: the smallest call, where launch latency counts.
        dict(name="attn-decode-1x1027-h32", op="attn", q_heads=32, kv_heads=32, dim=128, page=256, bits=16, group=128,
             q_lens="1", kv_lens="1027", window=0),
        # A serving batch of 32 conversations of many lengths (one to 8191
        # tokens) on the grouped-head model, one new token each.
        dict(name="attn-decode-32xragged-h64kv8", op="attn", q_heads=64, kv_heads=8, dim=128, page=256, bits=16,
             group=128, q_lens="1x32",
             kv_lens="1,8191,4096,517,2049,7003,300,6144,1025,33,5001,2750,8000,64,3500,4097,17,7777,1600,129,2222,"
                     "6500,900,4800,255,5555,3001,1234,7400,420,3900,2048", window=0),
        # Four long documents in a 4-bit cache, one new token each: the cache
        # format's purpose, and offsets past 32 bits of codes times heads.
        dict(name="attn-decode-4x64k-q4-h64kv8", op="attn", q_heads=64, kv_heads=8, dim=128, page=256, bits=4,
             group=32, q_lens="1x4", kv_lens="65536,40001,65000,52345", window=0),
        # A prompt of 8192 tokens on the grouped-head model in one chunk: the
        # largest call.
        dict(name="attn-prefill-8192-h64kv8", op="attn", q_heads=64, kv_heads=8, dim=128, page=256, bits=16, group=128,
             q_lens="8192", kv_lens="8192", window=0),
        # The next 511 tokens of a long prompt (chunked prefill) on the
        # 40-head model over an 8-bit cache.
        dict(name="attn-chunk-511at16k-q8-h40", op="attn", q_heads=40, kv_heads=40, dim=128, page=256, bits=8,
             group=128, q_lens="511", kv_lens="16384", window=0),
        # Continuous batching with a sliding window and small pages: prompts,
        # short drafts to verify and single tokens in one call, 64-wide heads.
        dict(name="attn-mixed-window-h32kv4-d64", op="attn", q_heads=32, kv_heads=4, dim=64, page=16, bits=16,
             group=64, q_lens="700,1,5,1,1333,1,8,1,1,257,1,4", kv_lens="700,2048,1000,3333,1500,77,4097,1,5000,257,"
             "900,12", window=1024),
        # The same layer's rotary step for 16 single tokens.
        dict(name="rope-append-16-h32", op="rope", tokens=16, q_heads=32, kv_heads=32, dim=128, rot=128,
             layout="half", page=256, bits=16, group=128, max_pos=4096),
        # A prompt's rotary step into an 8-bit cache: half of each head
        # rotated, neighbouring pairs, positions up to 128k.
        dict(name="rope-append-8191-q8-h64kv8", op="rope", tokens=8191, q_heads=64, kv_heads=8, dim=128, rot=64,
             layout="interleaved", page=64, bits=8, group=64, max_pos=131072),
        # The norm before a decode step's first layer: one token.
        dict(name="norm-1x4096", op="norm", tokens=1, hidden=4096, residual=True),
        # The same in a prompt of the largest model.
        dict(name="norm-8192x8192", op="norm", tokens=8192, hidden=8192, residual=True),
        # A conversation forks: the one partly filled page of each of 32 layers.
        dict(name="pages-fork-1x32", op="pages", layers=32, pool=8, moves=1, kv_heads=32, dim=128, page=64, bits=16,
             group=128),
        # The pool of a 4-bit cache is compacted.
        dict(name="pages-compact-151x16-q4", op="pages", layers=16, pool=320, moves=151, kv_heads=8, dim=128, page=256,
             bits=4, group=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = ((32, 32), (40, 40), (64, 8), (32, 4), (24, 8), (20, 4), (16, 1))


def _draw_cache(rng):
    bits = rng.choice((16, 16, 8, 6, 4))
    dim = rng.choice((64, 128, 128, 128, 256))
    groups = [g for g in (32, 64, 128) if dim % g == 0]
    return dict(bits=bits, dim=dim, group=rng.choice(groups), page=rng.choice((16, 32, 64, 128, 256)))


def draw(rng):
    kind = rng.choice(("decode", "decode", "chunk", "chunk", "rope", "norm", "pages"))
    if kind in ("decode", "chunk"):
        c = dict(op="attn", **_draw_cache(rng))
        c["q_heads"], c["kv_heads"] = rng.choice(_HEADS)
        per_token = 4 * c["kv_heads"] * c["dim"]
        if kind == "decode":
            n = _log_int(rng, 1, 64)
            cap = max(1, min(65536, int(1.2e9 / (per_token * n))))
            top = _log_int(rng, 1, cap)
            kv = [max(1, int(top * rng.random() + 0.5)) for _ in range(n - 1)] + [top]
            step = rng.choice((1, 1, 1, 2, 4, 7))
            q = [min(step, l) for l in kv]
        else:
            n = rng.choice((1, 1, 2, 5))
            top = _log_int(rng, 16, 8192 // n)
            past = _log_int(rng, 1, 16384) - 1
            while 4.0 * c["q_heads"] * c["dim"] * n * top * (past + 0.5 * top) > 1.0e12:
                past, top = past // 2, max(16, top - top // 4)
            q = [top] + [max(1, int(top * rng.random())) for _ in range(n - 1)]
            kv = [x + past for x in q]
        c["q_lens"] = ",".join(map(str, q))
        c["kv_lens"] = ",".join(map(str, kv))
        c["window"] = rng.choice((0, 0, 0, _log_int(rng, 1, 4096)))
        return c
    if kind == "rope":
        c = dict(op="rope", **_draw_cache(rng))
        c["q_heads"], c["kv_heads"] = rng.choice(_HEADS)
        c["tokens"] = _log_int(rng, 1, 8192 * 64 * 128 // (c["q_heads"] * c["dim"]) // 2)
        c["rot"] = rng.choice((c["dim"], c["dim"], c["dim"] // 2, c["dim"] // 4))
        c["layout"] = rng.choice(("half", "interleaved"))
        c["max_pos"] = max(c["tokens"], _log_int(rng, 64, 131072))
        return c
    if kind == "norm":
        hidden = rng.choice((64, 1000, 2048, 4096, 5120, 8192, _log_int(rng, 1, 16384)))
        return dict(op="norm", tokens=_log_int(rng, 1, min(65536, 8192 * 8192 // hidden)), hidden=hidden,
                    residual=rng.random() < 0.7)
    c = dict(op="pages", **_draw_cache(rng))
    c["kv_heads"] = rng.choice((1, 4, 8, 32))
    c["layers"] = rng.choice((1, 2, 16, 32, 80))
    one = 2 * c["kv_heads"] * c["page"] * c["dim"] * 2 * c["layers"]
    c["moves"] = _log_int(rng, 1, max(1, min(512, int(4e8 / one))))
    c["pool"] = 2 * c["moves"] + rng.randrange(1, 8)
    return c


# ---------------------------------------------------------------- inputs

def _lens(text):
    out = []
    for part in text.split(","):
        a, _, n = part.partition("x")
        out += [int(a)] * (int(n) if n else 1)
    return out


def _spread(gen, shape, dim):
    """Key/value-like rows: N(0, 1) with a magnitude per channel (a few channels several times larger)."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    mag = torch.exp(0.4 * torch.randn(dim, generator=gen, device="cuda"))
    return x.mul_(mag.to(torch.float16))


def _encode(x, bits, group):
    """float16 [..., D] -> (int32 words [..., D * bits / 32], float16 scales [..., D / group])."""
    half = 1 << (bits - 1)
    D = x.shape[-1]
    xf = x.float().view(*x.shape[:-1], D // group, group)
    s = (xf.abs().amax(-1) / float(half - 1)).to(torch.float16)
    sf = s.float().unsqueeze(-1)
    r = torch.where(sf > 0, torch.round(xf / torch.where(sf > 0, sf, torch.ones_like(sf))), torch.zeros_like(xf))
    q = (r.clamp(-half, half - 1) + half).to(torch.int64).view(*x.shape[:-1], D)
    return _pack(q, bits), s


def _pack(q, bits):
    """Codes int64 [..., D] -> words: runs of 16 codes fill bits / 2 words."""
    D = q.shape[-1]
    g = q.view(*q.shape[:-1], D // 16, 16)
    words = []
    for w in range(bits // 2):
        acc = torch.zeros_like(g[..., 0])
        for i in range(16):
            sh = i * bits - 32 * w
            if -bits < sh < 32:
                acc |= (g[..., i] << sh) if sh >= 0 else (g[..., i] >> -sh)
        acc &= 0xFFFFFFFF
        words.append(torch.where(acc >= 1 << 31, acc - (1 << 32), acc).to(torch.int32))
    return torch.stack(words, -1).reshape(*q.shape[:-1], D * bits // 32)


def _codes(words, D, bits):
    """Words -> codes int32 [..., D]."""
    w = (words.to(torch.int64) & 0xFFFFFFFF).view(*words.shape[:-1], D // 16, bits // 2)
    out = []
    for i in range(16):
        k, sh = divmod(i * bits, 32)
        v = w[..., k] >> sh
        if sh + bits > 32:
            v = v | (w[..., k + 1] << (32 - sh))
        out.append((v & ((1 << bits) - 1)).to(torch.int32))
    return torch.stack(out, -1).reshape(*words.shape[:-1], D)


def _values(words, scales, D, bits, group):
    """float16 values that codes and scales stand for."""
    q = _codes(words, D, bits).float() - float(1 << (bits - 1))
    q = q.view(*words.shape[:-1], D // group, group) * scales.float().unsqueeze(-1)
    return q.view(*words.shape[:-1], D).to(torch.float16)


def _pools(gen, case, pages):
    """Pools of rows as _spread makes them, encoded for 8, 6 and 4 bits."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    p = {}
    for name in ("k", "v"):
        x = _spread(gen, shape, case["dim"])
        if case["bits"] == 16:
            p[name] = x
            continue
        words, scales = [], []
        for part in x.split(max(1, (1 << 24) // x[0].numel())):
            w, s = _encode(part, case["bits"], case["group"])
            words.append(w)
            scales.append(s)
        p[name], p[name + "_scales"] = torch.cat(words), torch.cat(scales)
    return p


def _layer_pools(gen, case):
    """Every layer's pools in one tensor of each kind, [layers][pages]...: page
    copies move bits, so the quantized ones hold any words and scales."""
    shape = (case["layers"], case["pool"], case["kv_heads"], case["page"])
    p = {}
    for name in ("k", "v"):
        if case["bits"] == 16:
            p[name] = _spread(gen, shape + (case["dim"],), case["dim"])
            continue
        p[name] = torch.randint(-2 ** 31, 2 ** 31, shape + (case["dim"] * case["bits"] // 32,), generator=gen,
                                device="cuda", dtype=torch.int32)
        p[name + "_scales"] = torch.rand(shape + (case["dim"] // case["group"],), generator=gen, device="cuda",
                                         dtype=torch.float16)
    return p


def _cache(case, pools):
    import dequant_matmul_gptq_amd as dq
    return dq.KVCache(pools["k"], pools["v"], pools.get("k_scales"), pools.get("v_scales"), head_dim=case["dim"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=case)
    op = case["op"]
    if op == "attn":
        ql, kl = _lens(case["q_lens"]), _lens(case["kv_lens"])
        P = case["page"]
        need = [-(-l // P) for l in kl]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((len(kl), max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        st["pools"] = _pools(gen, case, pages)
        st["table"] = table
        st["q"] = torch.randn((sum(ql), case["q_heads"], case["dim"]), generator=gen, device="cuda",
                              dtype=torch.float16)
        st["kv_len"] = torch.tensor(kl, dtype=torch.int32, device="cuda")
        starts = [0]
        for n in ql:
            starts.append(starts[-1] + n)
        st["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        st["q_lens"], st["kv_lens"] = ql, kl
        if own:
            import dequant_matmul_gptq_amd as dq
            st["cache"] = _cache(case, st["pools"])
            st["out"] = torch.empty_like(st["q"])
            st["workspace"] = dq.paged_attention_workspace(st["cache"], sum(ql), case["q_heads"], len(ql), max(ql),
                                                           max(kl), "cuda", window=case["window"])
    elif op == "rope":
        T, P = case["tokens"], case["page"]
        pages = -(-T // P) + 2
        st["pools"] = _pools(gen, case, pages)
        for name, heads in (("q", case["q_heads"]), ("k", case["kv_heads"]), ("v", case["kv_heads"])):
            st[name] = _spread(gen, (T, heads, case["dim"]), case["dim"])
        first = int(torch.randint(0, case["max_pos"] - T + 1, (1,), generator=gen, device="cuda"))
        st["positions"] = torch.arange(first, first + T, device="cuda", dtype=torch.int32)
        order = torch.randperm(pages, generator=gen, device="cuda")
        i = torch.arange(T, device="cuda")
        st["slots"] = (order[i // P] * P + i % P).to(torch.int32)
        st["table"] = _rope_rows(case)
        st["q_out"] = torch.empty_like(st["q"])
        if own:
            st["cache"] = _cache(case, st["pools"])
    elif op == "norm":
        shape = (case["tokens"], case["hidden"])
        st["x"] = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
        if case["residual"]:
            st["r"] = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16) * 4
        st["w"] = (1 + 0.2 * torch.randn(case["hidden"], generator=gen, device="cuda")).to(torch.float16)
        st["y"], st["h"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
    else:
        st["pools"] = _layer_pools(gen, case)
        order = torch.randperm(case["pool"], generator=gen, device="cuda")[:2 * case["moves"]]
        st["pairs"] = order.view(case["moves"], 2).to(torch.int32).contiguous()
        if own:
            st["caches"] = [_cache(case, {n: t[i] for n, t in st["pools"].items()}) for i in range(case["layers"])]
    return st


def _rope_rows(case):
    """(cos, sin) pairs float32 [max_pos][rot / 2][2], from 64-bit angles."""
    half = case["rot"] // 2
    inv = ROPE_BASE ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    ang = torch.arange(case["max_pos"], dtype=torch.float64, device="cuda").unsqueeze(1) * inv
    return torch.stack((torch.cos(ang), torch.sin(ang)), -1).float()


# ---------------------------------------------------------------- one pass

def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import dequant_matmul_gptq_amd as dq
    case = st["case"]
    op = case["op"]
    if op == "attn":
        return dq.paged_attention(st["cache"], st["q"], st["table"], st["kv_len"], st["q_start"],
                                  max_q_len=max(st["q_lens"]), max_kv_len=max(st["kv_lens"]), window=case["window"],
                                  out=st["out"], workspace=st["workspace"])
    if op == "rope":
        layout = dq.ROPE_HALF if case["layout"] == "half" else dq.ROPE_INTERLEAVED
        dq.rope_append(st["cache"], st["q"], st["k"], st["v"], st["positions"], st["slots"], st["table"],
                       layout=layout, q_out=st["q_out"])
        p = st["pools"]
        if case["bits"] == 16:
            return st["q_out"], p["k"], p["v"]
        return (st["q_out"],) + tuple(dq.kv_dequant(p[n], p[n + "_scales"], case["dim"], case["bits"], case["group"])
                                      for n in ("k", "v"))
    if op == "norm":
        y = dq.rms_norm(st["x"], st["w"], residual=st.get("r"), out=st["y"],
                        residual_out=st["h"] if case["residual"] else None)
        return (y, st["h"]) if case["residual"] else y
    dq.copy_pages(st["caches"], st["pairs"])
    return list(st["pools"].values())          # as stored: words and scales, bit for bit


def _rows(p, name, case, table, L):
    """float32 [kv_heads][L][dim]: the first L rows behind one block table row."""
    idx = table[:-(-L // case["page"])].long()
    if case["bits"] == 16:
        x = p[name][idx].float()
    else:
        x = _values(p[name][idx], p[name + "_scales"][idx], case["dim"], case["bits"], case["group"]).float()
    return x.transpose(0, 1).reshape(case["kv_heads"], -1, case["dim"])[:, :L]


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "attn":
        return _plain_attention(st)
    if op == "rope":
        return _plain_rope(st)
    if op == "norm":
        if case["residual"]:
            h = (st["x"].float() + st["r"].float()).to(torch.float16)
        else:
            h = st["x"]
        hf = h.float()
        y = (hf / torch.sqrt((hf * hf).mean(-1, keepdim=True) + 1e-5) * st["w"].float()).to(torch.float16)
        return (y, h) if case["residual"] else y
    src, dst = st["pairs"][:, 0].long(), st["pairs"][:, 1].long()
    for t in st["pools"].values():
        t[:, dst] = t[:, src]
    return list(st["pools"].values())          # as stored: words and scales, bit for bit


def _plain_attention(st):
    case, p = st["case"], st["pools"]
    Hq, Hk, D = case["q_heads"], case["kv_heads"], case["dim"]
    G = Hq // Hk
    scale = 1.0 / math.sqrt(D)
    out = torch.empty_like(st["q"])
    at = 0
    for b, (n, L) in enumerate(zip(st["q_lens"], st["kv_lens"])):
        k = _rows(p, "k", case, st["table"][b], L)
        v = _rows(p, "v", case, st["table"][b], L)
        pos = torch.arange(L - n, L, device="cuda").unsqueeze(1)
        t = torch.arange(L, device="cuda").unsqueeze(0)
        masked = t > pos
        if case["window"]:
            masked |= t <= pos - case["window"]
        q = st["q"][at:at + n].float().view(n, Hk, G, D).permute(1, 2, 0, 3)
        for c in range(Hk):
            s = torch.matmul(q[c].reshape(G * n, D), k[c].t()).view(G, n, L).mul_(scale)
            s.masked_fill_(masked, -math.inf)
            s = torch.exp(s.sub_(s.amax(-1, keepdim=True)))
            s /= s.sum(-1, keepdim=True)
            o = torch.matmul(s.view(G * n, L), v[c]).view(G, n, D)
            out[at:at + n, c * G:(c + 1) * G] = o.transpose(0, 1).to(torch.float16)
        at += n
    return out


def _rotate(x, cs, rot, layout):
    """Rotated copy of x [T][H][D] in the precision of x and cs [T][rot / 2][2]."""
    c, s = cs[..., 0].unsqueeze(1), cs[..., 1].unsqueeze(1)
    y = x.clone()
    if layout == "half":
        a, b = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        a, b = slice(0, rot, 2), slice(1, rot, 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _plain_rope(st):
    case, p = st["case"], st["pools"]
    cs = st["table"][st["positions"].long()]
    st["q_out"].copy_(_rotate(st["q"].float(), cs, case["rot"], case["layout"]))
    k = _rotate(st["k"].float(), cs, case["rot"], case["layout"]).to(torch.float16)
    pg, off = st["slots"].long() // case["page"], st["slots"].long() % case["page"]
    for name, x in (("k", k), ("v", st["v"])):
        if case["bits"] == 16:
            p[name][pg, :, off] = x
        else:
            p[name][pg, :, off], p[name + "_scales"][pg, :, off] = _encode(x, case["bits"], case["group"])
    if case["bits"] == 16:
        return st["q_out"], p["k"], p["v"]
    return (st["q_out"],) + tuple(_values(p[n], p[n + "_scales"], case["dim"], case["bits"], case["group"])
                                  for n in ("k", "v"))


# ---------------------------------------------------------------- bytes and operations

def _row_bytes(case):
    if case["bits"] == 16:
        return 2 * case["dim"]
    return case["dim"] * case["bits"] // 8 + 2 * case["dim"] // case["group"]


def work(case):
    op = case["op"]
    if op == "attn":
        D, w = case["dim"], case["window"]
        rows = pairs = 0
        for n, L in zip(_lens(case["q_lens"]), _lens(case["kv_lens"])):
            first = L - n
            if w:
                rows += L - max(0, first - w + 1)
                full = max(0, n - max(0, w - 1 - first))          # new tokens whose window is full
                m = n - full
                pairs += full * w + m * first + m * (m + 1) // 2
            else:
                rows += L
                pairs += n * first + n * (n + 1) // 2
        T = sum(_lens(case["q_lens"]))
        return {"bytes": rows * case["kv_heads"] * 2 * _row_bytes(case) + 2 * T * case["q_heads"] * D * 2,
                "flops": 4 * D * case["q_heads"] * pairs}
    if op == "rope":
        T, D = case["tokens"], case["dim"]
        b = T * (2 * case["q_heads"] * D * 2 + 2 * case["kv_heads"] * D * 2 + 4 * case["rot"])
        b += T * case["kv_heads"] * 2 * _row_bytes(case)
        if case["bits"] != 16:                     # the pools come back as the values they stand for
            rows = (-(-T // case["page"]) + 2) * case["page"]
            b += rows * case["kv_heads"] * 2 * (_row_bytes(case) + 2 * D)
        return {"bytes": b, "flops": 3 * T * case["rot"] * (case["q_heads"] + case["kv_heads"])}
    if op == "norm":
        n = case["tokens"] * case["hidden"]
        return {"bytes": (8 if case["residual"] else 4) * n + 2 * case["hidden"], "flops": 5 * n}
    return {"bytes": 2 * case["moves"] * case["layers"] * case["kv_heads"] * case["page"] * 2 * _row_bytes(case),
            "flops": 0}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = st["x"].double()
        if case["residual"]:
            h = (h + st["r"].double()).to(torch.float16).double()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-5) * st["w"].double()
        return (y, h) if case["residual"] else y
    if op == "pages":
        pools = list(st["pools"].values())
        for src, dst in st["pairs"].tolist():
            for t in pools:
                t[:, dst].copy_(t[:, src])
        return pools
    if op == "rope":
        return _exact_rope(st)
    if work(case)["flops"] > 4e12:
        return None
    return _exact_attention(st)


def _stored(p, name, case):
    """float64 pool: the values a whole pool stands for."""
    if case["bits"] == 16:
        return p[name].double()
    bits, D = case["bits"], case["dim"]
    words = p[name].long() & 0xFFFFFFFF
    i = torch.arange(D, device="cuda") * bits
    lo = words[..., i // 32] >> (i % 32)
    nxt = words[..., torch.clamp(i // 32 + 1, max=words.shape[-1] - 1)] << (32 - i % 32)
    q = (torch.where(i % 32 + bits > 32, lo | nxt, lo) & ((1 << bits) - 1)).double() - 2.0 ** (bits - 1)
    s = p[name + "_scales"].double().repeat_interleave(case["group"], -1)
    return (q * s).to(torch.float16).double()


def _exact_attention(st):
    case = st["case"]
    Hq, Hk, D, P, w = (case[x] for x in ("q_heads", "kv_heads", "dim", "page", "window"))
    res = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, L) in enumerate(zip(st["q_lens"], st["kv_lens"])):
        t = torch.arange(L, device="cuda")
        page = st["table"][b].long()[t // P]
        for c in range(Hk):
            part = {}
            for name in ("k", "v"):
                sub = {name: st["pools"][name][:, c]}
                if case["bits"] != 16:
                    sub[name + "_scales"] = st["pools"][name + "_scales"][:, c]
                sub = {key: x[page, t % P] for key, x in sub.items()}
                part[name] = _stored(sub, name, case)
            for h in range(c * (Hq // Hk), (c + 1) * (Hq // Hk)):
                for i in range(0, n, 2048):
                    m = min(2048, n - i)
                    pos = torch.arange(L - n + i, L - n + i + m, device="cuda")
                    z = st["q"][at + i:at + i + m, h].double() @ part["k"].T / math.sqrt(D)
                    see = t[None, :] <= pos[:, None]
                    if w > 0:
                        see &= pos[:, None] - t[None, :] < w
                    z = torch.where(see, z, torch.full_like(z, -math.inf))
                    e = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
                    res[at + i:at + i + m, h] = e @ part["v"]
        at += n
    return res


def _exact_rope(st):
    case, p = st["case"], st["pools"]
    T, P, r, D = case["tokens"], case["page"], case["rot"], case["dim"]
    cs = st["table"].double()[st["positions"].long()]
    z = torch.complex(cs[..., 0], cs[..., 1]).unsqueeze(1)
    done = {}
    for name in ("q", "k"):
        x = st[name].double()
        head = x[..., :r]
        if case["layout"] == "half":
            u = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) * z
            head = torch.cat((u.real, u.imag), -1)
        else:
            u = torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2).contiguous()) * z
            head = torch.view_as_real(u).reshape(head.shape)
        done[name] = torch.cat((head, x[..., r:]), -1)
    out = [done["q"]]
    slot = st["slots"].long()
    for name, x in (("k", done["k"]), ("v", st["v"].double())):
        if case["bits"] != 16:
            half = 1 << (case["bits"] - 1)
            x = x.to(torch.float16).double().reshape(T, -1, D // case["group"], case["group"])
            s = (x.abs().amax(-1, keepdim=True) / (half - 1)).to(torch.float16).double()
            q = torch.where(s > 0, torch.round(x / s.clamp(min=1e-30)), torch.zeros_like(x)).clamp(-half, half - 1)
            x = (q * s).to(torch.float16).double().reshape(T, -1, D)
        pool = _stored(p, name, case)
        pool[slot // P, :, slot % P] = x
        out.append(pool)
    return tuple(out)
