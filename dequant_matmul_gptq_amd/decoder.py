"""Binding of the operators between a decoder's linear layers: the paged
key/value cache, rotary positions, attention, page copies and the norm, and of
what is read off the head's logits (argument marshalling; the one computation
here is the host-made table of rotary angles). Checks, streams and errors are
those of the other calls: wrong tensors raise ValueError, a non-zero status
QlinearError.
"""

from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import numpy as np
import torch

from ._lib import _check, _dev, _ptr, lib, qlinear_kv_cache

ROPE_HALF = 0
ROPE_INTERLEAVED = 1

_F16, _F32, _I32, _U8 = torch.float16, torch.float32, torch.int32, torch.uint8

# These calls are short on the GPU (a few microseconds for one token), so the
# checks below are kept to a few attribute reads, and the stream is taken as
# the raw handle (0.1 us; a Stream object takes 2 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream if _raw_stream is None else _raw_stream(device)


# A call's GPU has to be the current one: a default stream's handle is 0 on all
# GPUs and means that of the current one. Where it is not, the call is made again
# with it.
_current_gpu = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

_INT_MAX = 2 ** 31 - 1


def _int32(*numbers):
    """The numbers as the C calls take them. ctypes would cut them to 32 bits; a
    bound (of a length, a window) past those is as good as the largest one, and
    a size or a negative number past them is refused as the largest or -1 is.
    Callers come here if the numbers' or, shifted by 31, is not 0."""
    return tuple(max(-1, min(n, _INT_MAX)) for n in numbers)


def _gpu_of(t: torch.Tensor, name: str) -> int:
    """The GPU that the call runs on, that of its operand t."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return device


def _operand(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device: int) -> int:
    """Check a contiguous operand on GPU `device` and return its pointer."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous():
        _dev(t, name, dtype, shape)
        raise ValueError(f"{name} must be on GPU {device}, got {t.device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, tokens: int | None, heads: int | None, dim: int | None, device: int):
    """Check a float16 [tokens][heads][dim] operand on GPU `device` whose tokens
    may be strided (a slice of a fused projection). Returns its pointer, shape
    and token stride."""
    if t.dtype is not _F16 or t.get_device() != device or t.dim() != 3:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if t.dtype is not _F16:
            raise ValueError(f"{name} must be {_F16}, got {t.dtype}")
        if t.dim() != 3:
            raise ValueError(f"{name} must be [tokens][heads][head_dim], got {tuple(t.shape)}")
        raise ValueError(f"{name} must be on GPU {device}, got {t.device}")
    T, h, d = t.shape
    if (tokens is not None and T != tokens) or (heads is not None and h != heads) or (dim is not None and d != dim):
        want = [n if v is None else v for n, v in (("tokens", tokens), ("heads", heads), ("head_dim", dim))]
        raise ValueError(f"{name} must be [{want[0]}][{want[1]}][{want[2]}], got {tuple(t.shape)}")
    st, sh, sd = t.stride()
    if T < 2 or h == 0 or d == 0:
        st = h * d
    if T > 0 and ((d > 1 and sd != 1) or (h > 1 and sh != d)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), T, h, d, st


class KVCache:
    """Key/value pools of one layer (wraps qlinear_kv_cache).

    k, v: float16 [num_pages][kv_heads][page_size][head_dim], or code words
    int32 [num_pages][kv_heads][page_size][head_dim * bits / 32] with scales
    float16 [num_pages][kv_heads][page_size][head_dim / group] (the rows of
    kv_quant; head_dim says how wide they are, and the width follows).
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: torch.Tensor | None = None,
                 v_scales: torch.Tensor | None = None, head_dim: int | None = None):
        if k.dim() != 4:
            raise ValueError("k must be [num_pages][kv_heads][page_size][...]")
        if (k_scales is None) != (v_scales is None):
            raise ValueError("k_scales and v_scales go together")
        pages, heads, page, width = (int(n) for n in k.shape)
        if k_scales is None:
            if head_dim is not None and int(head_dim) != width:
                raise ValueError(f"k must be [num_pages][kv_heads][page_size][{head_dim}]")
            self.head_dim, self.bits, self.group = width, 16, 0
            dtype = torch.float16
        else:
            if head_dim is None or head_dim < 1 or 32 * width % head_dim != 0:
                raise ValueError("a quantized cache needs head_dim, and its rows head_dim * bits / 32 words")
            if k_scales.dim() != 4 or k_scales.shape[3] < 1 or head_dim % k_scales.shape[3] != 0:
                raise ValueError("k_scales must be [num_pages][kv_heads][page_size][head_dim / group]")
            self.head_dim, self.bits = int(head_dim), 32 * width // int(head_dim)
            self.group = self.head_dim // int(k_scales.shape[3])
            dtype = torch.int32
            for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
                _dev(t, name, torch.float16, (pages, heads, page, self.head_dim // self.group))
        _dev(k, "k", dtype)
        _dev(v, "v", dtype, tuple(k.shape))
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.num_pages, self.kv_heads, self.page_size = pages, heads, page
        self.c = qlinear_kv_cache(_ptr(k), _ptr(v), _ptr(k_scales), _ptr(v_scales), pages, page, heads, self.head_dim,
                                  self.bits, self.group)
        self.ref, self.raw = ctypes.byref(self.c), bytes(self.c)
        self.device = k.get_device()
        for name, t in (("v", v), ("k_scales", k_scales), ("v_scales", v_scales)):
            if t is not None and t.get_device() != self.device:
                raise ValueError(f"{name} must be on GPU {self.device}, got {t.device}")

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, head_dim: int, page_size: int = 256, bits: int = 16,
              group: int = 32, device="cuda") -> "KVCache":
        """Pools of the given shape, not initialized (slots that no token has
        been appended to are never used). `group` is for bits 8, 6 and 4."""
        lead = (num_pages, kv_heads, page_size)
        if bits == 16:
            return cls(*(torch.empty(lead + (head_dim,), dtype=torch.float16, device=device) for _ in range(2)))
        if bits not in (4, 6, 8) or group not in (32, 64, 128) or head_dim % group != 0:
            raise ValueError("bits must be 16, 8, 6 or 4, group 32, 64 or 128 and a divisor of head_dim")
        kv = [torch.empty(lead + (head_dim * bits // 32,), dtype=torch.int32, device=device) for _ in range(2)]
        s = [torch.empty(lead + (head_dim // group,), dtype=torch.float16, device=device) for _ in range(2)]
        return cls(*kv, *s, head_dim=head_dim)


# ---------------------------------------------------------------- rotary positions

def rope_table(max_pos: int, rot_dim: int, base: float = 10000.0, scaling: dict | None = None,
               device="cpu") -> torch.Tensor:
    """(cos, sin) of every position and pair, float32 [max_pos][rot_dim / 2][2],
    computed in 64 bits: angle p * f_i with f_i = base^(-2 i / rot_dim), changed
    for long contexts by `scaling` (type and its numbers):

    - linear, factor: f_i / factor (positions compressed).
    - ntk, factor: base * factor^(rot_dim / (rot_dim - 2)) (the lowest
      frequency is divided by factor, the highest kept).
    - bands, factor, original (trained length), low, high: with w_i = original *
      f_i / (2 pi) turns over the trained length, f_i / factor for w_i < low,
      f_i for w_i > high, and linear in w_i between the two.
    - yarn, factor, original, beta_fast (32), beta_slow (1), attention (None):
      between f_i / factor and f_i by a ramp over i, from the pair that makes
      beta_fast turns over the trained length (rounded down) to that of
      beta_slow (rounded up); cos and sin are multiplied by `attention`,
      0.1 ln(factor) + 1 if it is None.
    """
    if max_pos < 1 or rot_dim < 2 or rot_dim % 2 != 0 or not base > 0:
        raise ValueError("rope_table needs max_pos >= 1, an even rot_dim >= 2 and a positive base")
    i = np.arange(rot_dim // 2, dtype=np.float64)
    sc = dict(scaling or {"type": "none"})
    kind = sc.pop("type", None)
    need = {"none": set(), "linear": {"factor"}, "ntk": {"factor"}, "bands": {"factor", "original", "low", "high"},
            "yarn": {"factor", "original"}}
    optional = {"yarn": {"beta_fast", "beta_slow", "attention"}}
    if kind not in need or not need[kind] <= set(sc) <= need[kind] | optional.get(kind, set()):
        raise ValueError(f"unknown rotary scaling {scaling!r}")
    factor = float(sc.get("factor", 1.0))
    if not factor >= 1.0:
        raise ValueError("the scaling factor must be at least 1")
    if kind == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim >= 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-2.0 * i / rot_dim)
    amp = 1.0
    if kind == "linear":
        f = f / factor
    elif kind == "bands":
        low, high = float(sc["low"]), float(sc["high"])
        if not 0 < low < high:
            raise ValueError("bands scaling needs 0 < low < high")
        keep = np.clip((float(sc["original"]) * f / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
        f = f * keep + f / factor * (1 - keep)
    elif kind == "yarn":
        def pair_of(turns):
            return rot_dim * math.log(float(sc["original"]) / (turns * 2 * math.pi)) / (2 * math.log(base))
        first = max(math.floor(pair_of(float(sc.get("beta_fast", 32.0)))), 0)
        last = min(math.ceil(pair_of(float(sc.get("beta_slow", 1.0)))), rot_dim - 1)
        ramp = np.clip((i - first) / max(last - first, 1e-3), 0.0, 1.0)
        f = f / factor * ramp + f * (1 - ramp)
        amp = sc.get("attention")
        amp = 0.1 * math.log(factor) + 1.0 if amp is None else float(amp)
    out = np.empty((max_pos, rot_dim // 2, 2), dtype=np.float32)
    step = max(1, (1 << 22) // (rot_dim // 2))
    for p in range(0, max_pos, step):
        ang = np.arange(p, min(p + step, max_pos), dtype=np.float64)[:, None] * f
        out[p:p + step, :, 0] = np.cos(ang) * amp
        out[p:p + step, :, 1] = np.sin(ang) * amp
    return torch.from_numpy(out).to(device)


def _rope_operands(table: torch.Tensor, positions: torch.Tensor, tokens: int, device: int):
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("table must be [positions][rot_dim / 2][2]")
    rows, half, _ = table.shape
    return (_operand(positions, "positions", _I32, (tokens,), device),
            _operand(table, "table", _F32, (rows, half, 2), device), rows, 2 * half)


def _norm_weight(w: torch.Tensor | None, name: str, heads: int, dim: int, device: int):
    """Pointer and number of rows of a norm's weight, [head_dim] or [heads][head_dim]."""
    if w is None:
        return None, 1
    if w.dim() == 1:
        return _operand(w, name, _F16, (dim,), device), 1
    return _operand(w, name, _F16, (heads, dim), device), heads


def rope(x: torch.Tensor, positions: torch.Tensor | None, table: torch.Tensor | None, layout: int = ROPE_HALF,
         out: torch.Tensor | None = None, norm: torch.Tensor | None = None, eps: float = 1e-6) -> torch.Tensor:
    """x float16 [tokens][heads][head_dim] (token stride free) rotated to the
    positions (int32 [tokens]) by the table of rope_table. out may be x.

    norm float16 [head_dim] or [heads][head_dim]: each head's row is first
    x / sqrt(mean(x^2) + eps) * norm, in the same pass (table None: that alone).
    """
    dev = _gpu_of(x, "x")
    if _current_gpu() != dev:
        with torch.cuda.device(dev):
            return rope(x, positions, table, layout, out, norm, eps)
    xp, T, H, D, xs = _rows(x, "x", None, None, None, dev)
    pos = tab = None
    rows = rot = 0
    if table is not None:
        if positions is None:
            raise ValueError("a table needs positions")
        pos, tab, rows, rot = _rope_operands(table, positions, T, dev)
    elif norm is None:
        raise ValueError("a call without a table needs a norm")
    wp, wh = _norm_weight(norm, "norm", H, D, dev)
    if out is None:
        out = torch.empty((T, H, D), dtype=_F16, device=x.device)
    op, _, _, _, ost = _rows(out, "out", T, H, D, dev)
    if (T | H | D | rows | rot) >> 31:
        T, H, D, rows, rot, wh = _int32(T, H, D, rows, rot, wh)
    if norm is None:
        _check(lib().qlinear_rope(xp, xs, T, H, D, pos, tab, rows, rot, layout, op, ost, _stream(dev)), "qlinear_rope")
    else:
        _check(lib().qlinear_norm_rope(xp, xs, T, H, D, wp, wh, eps, pos, tab, rows, rot, layout, op, ost,
                                       _stream(dev)), "qlinear_norm_rope")
    return out


def rope_append(cache: KVCache, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                positions: torch.Tensor | None, slots: torch.Tensor, table: torch.Tensor | None,
                layout: int = ROPE_HALF, q_out: torch.Tensor | None = None, q_norm: torch.Tensor | None = None,
                k_norm: torch.Tensor | None = None, eps: float = 1e-6) -> torch.Tensor | None:
    """Rotate q [tokens][q_heads][head_dim] (returned; q_out may be q) and k
    [tokens][kv_heads][head_dim] to the positions, and write k and v to the
    cache's slots (int32 [tokens]: page * page_size + place in the page,
    negative = not appended). table None: no rotation. q None: only the append.
    q_norm, k_norm: norms of their heads before the rotation, as in rope.
    """
    dev, D, Hk = cache.device, cache.head_dim, cache.kv_heads
    if _current_gpu() != dev:
        with torch.cuda.device(dev):
            return rope_append(cache, q, k, v, positions, slots, table, layout, q_out, q_norm, k_norm, eps)
    kp, T, _, _, ks = _rows(k, "k", None, Hk, D, dev)
    vp, _, _, _, vs = _rows(v, "v", T, Hk, D, dev)
    sp = _operand(slots, "slots", _I32, (T,), dev)
    pos = tab = qp = op = None
    rows = rot = heads = qs = ost = 0
    if table is not None:
        if positions is None:
            raise ValueError("a table needs positions")
        pos, tab, rows, rot = _rope_operands(table, positions, T, dev)
    if q is not None:
        qp, _, heads, _, qs = _rows(q, "q", T, None, D, dev)
        if q_out is None:
            q_out = torch.empty((T, heads, D), dtype=_F16, device=q.device)
        op, _, _, _, ost = _rows(q_out, "q_out", T, heads, D, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    elif q_norm is not None:
        raise ValueError("q_norm without q")
    if (T | heads | rows | rot) >> 31:
        T, heads, rows, rot = _int32(T, heads, rows, rot)
    if q_norm is None and k_norm is None:
        _check(lib().qlinear_rope_append(cache.ref, qp, qs, heads, kp, ks, vp, vs, op, ost, T, pos, sp, tab, rows, rot,
                                         layout, _stream(dev)), "qlinear_rope_append")
        return q_out
    qn, qn_heads = _norm_weight(q_norm, "q_norm", heads, D, dev)
    kn, kn_heads = _norm_weight(k_norm, "k_norm", Hk, D, dev)
    _check(lib().qlinear_norm_rope_append(cache.ref, qp, qs, heads, kp, ks, vp, vs, op, ost, T, qn, qn_heads, kn,
                                          kn_heads, eps, pos, sp, tab, rows, rot, layout, _stream(dev)),
           "qlinear_norm_rope_append")
    return q_out


# ---------------------------------------------------------------- attention

def paged_attention_workspace_bytes(cache: KVCache, tokens: int, q_heads: int, batch: int, max_q_len: int,
                                    max_kv_len: int, window: int = 0, sinks: int = 0) -> int:
    n = ctypes.c_size_t(0)
    sizes = _int32(int(tokens), int(q_heads), int(batch), int(max_q_len), int(max_kv_len), int(window))
    if sinks:
        _check(lib().qlinear_paged_attention_sinks_workspace_bytes(cache.ref, *sizes, *_int32(int(sinks)),
                                                                   ctypes.byref(n)),
               "qlinear_paged_attention_sinks_workspace_bytes")
    else:
        _check(lib().qlinear_paged_attention_workspace_bytes(cache.ref, *sizes, ctypes.byref(n)),
               "qlinear_paged_attention_workspace_bytes")
    return int(n.value)


def paged_attention_workspace(cache: KVCache, tokens: int, q_heads: int, batch: int, max_q_len: int, max_kv_len: int,
                              device, window: int = 0, sinks: int = 0) -> torch.Tensor:
    """A paged_attention workspace for calls of up to these sizes with the same
    q_heads, window and sinks (scratch: needs no initialization; calls that may
    overlap in time must not share one)."""
    n = paged_attention_workspace_bytes(cache, tokens, q_heads, batch, max_q_len, max_kv_len, window, sinks)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def paged_attention(cache: KVCache, q: torch.Tensor, block_table: torch.Tensor, kv_len: torch.Tensor,
                    q_start: torch.Tensor | None = None, max_q_len: int | None = None,
                    max_kv_len: int | None = None, scale: float | None = None, window: int = 0,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    sinks: int = 0) -> torch.Tensor:
    """Causal attention of each sequence's new tokens over its cached ones (the
    new ones among them, appended before the call).

    q float16 [tokens][q_heads][head_dim] (token stride free); block_table
    int32 [batch][width], a sequence's pages in order; kv_len int32 [batch],
    tokens in the cache; q_start int32 [batch + 1], sequence b's rows of q are
    q_start[b] .. q_start[b + 1] - 1 (None: tokens / batch rows each). window
    w > 0: a token sees the w last positions up to its own, and with sinks the
    sequence's first `sinks` tokens too. scale: None = head_dim^-0.5. max_q_len
    and max_kv_len bound the lengths for the launch plan (None: tokens, width *
    page_size); lengths stay on the device. Returns out float16
    [tokens][q_heads][head_dim]; a token that sees nothing gets zeros.
    """
    dev, D = cache.device, cache.head_dim
    if _current_gpu() != dev:
        with torch.cuda.device(dev):
            return paged_attention(cache, q, block_table, kv_len, q_start, max_q_len, max_kv_len, scale, window, out,
                                   workspace, sinks)
    qp, T, H, _, qs = _rows(q, "q", None, None, D, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch][width]")
    B, W = block_table.shape
    tp = _operand(block_table, "block_table", _I32, (B, W), dev)
    lp = _operand(kv_len, "kv_len", _I32, (B,), dev)
    sp = None if q_start is None else _operand(q_start, "q_start", _I32, (B + 1,), dev)
    if max_q_len is None:
        max_q_len = T if q_start is not None or B == 0 else T // B
    if max_kv_len is None:
        max_kv_len = W * cache.page_size
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty((T, H, D), dtype=_F16, device=q.device)
    op = _operand(out, "out", _F16, (T, H, D), dev)
    if workspace is None:
        workspace = paged_attention_workspace(cache, T, H, B, max_q_len, max_kv_len, q.device, window, sinks)
    n = workspace.numel()
    wp = _operand(workspace, "workspace", _U8, (n,), dev)
    if (T | H | B | W | max_q_len | max_kv_len | window | sinks) >> 31:
        T, H, B, W, max_q_len, max_kv_len, window, sinks = _int32(T, H, B, W, max_q_len, max_kv_len, window, sinks)
    if sinks:
        _check(lib().qlinear_paged_attention_sinks(cache.ref, qp, qs, T, H, B, sp, lp, tp, W, max_q_len, max_kv_len,
                                                   scale, window, sinks, op, wp, n, _stream(dev)),
               "qlinear_paged_attention_sinks")
    else:
        _check(lib().qlinear_paged_attention(cache.ref, qp, qs, T, H, B, sp, lp, tp, W, max_q_len, max_kv_len, scale,
                                             window, op, wp, n, _stream(dev)), "qlinear_paged_attention")
    return out


def paged_attention_shared_workspace_bytes(cache: KVCache, tokens: int, q_heads: int, batch: int, max_q_len: int,
                                           max_kv_len: int, groups: int, max_shared_len: int) -> int:
    n = ctypes.c_size_t(0)
    sizes = _int32(int(tokens), int(q_heads), int(batch), int(max_q_len), int(max_kv_len), int(groups),
                   int(max_shared_len))
    _check(lib().qlinear_paged_attention_shared_workspace_bytes(cache.ref, *sizes, ctypes.byref(n)),
           "qlinear_paged_attention_shared_workspace_bytes")
    return int(n.value)


def paged_attention_shared_workspace(cache: KVCache, tokens: int, q_heads: int, batch: int, max_q_len: int,
                                     max_kv_len: int, groups: int, max_shared_len: int, device) -> torch.Tensor:
    """A paged_attention_shared workspace for calls of up to these sizes with
    the same q_heads, whatever max_shared_len (scratch: needs no initialization;
    calls that may overlap in time must not share one)."""
    n = paged_attention_shared_workspace_bytes(cache, tokens, q_heads, batch, max_q_len, max_kv_len, groups,
                                               max_shared_len)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def paged_attention_shared(cache: KVCache, q: torch.Tensor, block_table: torch.Tensor, kv_len: torch.Tensor,
                           shared_len: torch.Tensor, shared_start: torch.Tensor | None = None,
                           q_start: torch.Tensor | None = None, max_q_len: int | None = None,
                           max_kv_len: int | None = None, max_shared_len: int | None = None,
                           scale: float | None = None, out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None) -> torch.Tensor:
    """paged_attention for sequences that share their first tokens, as forks of
    one sequence do: those are read once for all of a group's rows.

    Group g is the sequences shared_start[g] .. shared_start[g + 1] - 1 (int32
    [groups + 1]; None: one group of all), whose first shared_len[g] tokens
    (int32 [groups]; PagePool.shared_tokens counts them) are the same slots of
    the cache: at most each one's tokens before its new ones. Sequences of no
    group share nothing. max_shared_len bounds shared_len (None: width *
    page_size); it has no effect so far, the launch plan goes by max_kv_len. The
    rest is as for paged_attention, which does as well for two branches, short
    prefixes, and prompts of many new tokens.
    """
    dev, D = cache.device, cache.head_dim
    if _current_gpu() != dev:
        with torch.cuda.device(dev):
            return paged_attention_shared(cache, q, block_table, kv_len, shared_len, shared_start, q_start, max_q_len,
                                          max_kv_len, max_shared_len, scale, out, workspace)
    qp, T, H, _, qs = _rows(q, "q", None, None, D, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch][width]")
    B, W = block_table.shape
    tp = _operand(block_table, "block_table", _I32, (B, W), dev)
    lp = _operand(kv_len, "kv_len", _I32, (B,), dev)
    G = shared_len.numel()
    if shared_start is None and G != 1:
        raise ValueError("without shared_start all sequences are one group")
    gl = _operand(shared_len, "shared_len", _I32, (G,), dev)
    gs = None if shared_start is None else _operand(shared_start, "shared_start", _I32, (G + 1,), dev)
    sp = None if q_start is None else _operand(q_start, "q_start", _I32, (B + 1,), dev)
    if max_q_len is None:
        max_q_len = T if q_start is not None or B == 0 else T // B
    if max_kv_len is None:
        max_kv_len = W * cache.page_size
    if max_shared_len is None:
        max_shared_len = W * cache.page_size
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty((T, H, D), dtype=_F16, device=q.device)
    op = _operand(out, "out", _F16, (T, H, D), dev)
    if workspace is None:
        workspace = paged_attention_shared_workspace(cache, T, H, B, max_q_len, max_kv_len, G, max_shared_len, q.device)
    n = workspace.numel()
    wp = _operand(workspace, "workspace", _U8, (n,), dev)
    if (T | H | B | W | G | max_q_len | max_kv_len | max_shared_len) >> 31:
        T, H, B, W, G, max_q_len, max_kv_len, max_shared_len = _int32(T, H, B, W, G, max_q_len, max_kv_len,
                                                                      max_shared_len)
    _check(lib().qlinear_paged_attention_shared(cache.ref, qp, qs, T, H, B, sp, lp, tp, W, G, gs, gl, max_q_len,
                                                max_kv_len, max_shared_len, scale, op, wp, n, _stream(dev)),
           "qlinear_paged_attention_shared")
    return out


# ---------------------------------------------------------------- pages

def copy_pages(caches, pairs: torch.Tensor) -> None:
    """Page pairs[i][1] becomes a copy of page pairs[i][0] in every cache of
    `caches` (a model's layers, one shape); pairs int32 [moves][2]. No page may
    be a target and appear in another pair."""
    dev = pairs.get_device()
    if pairs.dim() != 2:
        raise ValueError("pairs must be [moves][2]")
    moves = pairs.shape[0]
    pp = _operand(pairs, "pairs", _I32, (moves, 2), dev)
    caches = list(caches)
    for c in caches:
        if c.device != dev:
            raise ValueError(f"pairs must be on the caches' GPU {c.device}, got {pairs.device}")
    if caches and _current_gpu() != dev:
        with torch.cuda.device(dev):
            return copy_pages(caches, pairs)
    # The structs side by side (ctypes' own array constructor takes 0.3 us each).
    arr = (qlinear_kv_cache * max(1, len(caches))).from_buffer_copy(
        b"".join([c.raw for c in caches]) or bytes(ctypes.sizeof(qlinear_kv_cache)))
    if moves >> 31:
        moves, = _int32(moves)
    _check(lib().qlinear_copy_pages(arr, len(caches), pp, moves, _stream(dev)), "qlinear_copy_pages")


# ---------------------------------------------------------------- norm

def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5, residual: torch.Tensor | None = None,
             out: torch.Tensor | None = None, residual_out: torch.Tensor | None = None) -> torch.Tensor:
    """y = h / sqrt(mean(h^2) + eps) * weight over the last dimension, with
    h = x + residual rounded to float16 (x without a residual) written to
    residual_out if it is given (it may be x or residual). out may be x."""
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    dev, shape = _gpu_of(x, "x"), x.shape
    if _current_gpu() != dev:
        with torch.cuda.device(dev):
            return rms_norm(x, weight, eps, residual, out, residual_out)
    K = shape[-1]
    xp = _operand(x, "x", _F16, shape, dev)
    wp = _operand(weight, "weight", _F16, (K,), dev)
    rp = None if residual is None else _operand(residual, "residual", _F16, shape, dev)
    if out is None:
        out = torch.empty_like(x)
    op = _operand(out, "out", _F16, shape, dev)
    hp = None if residual_out is None else _operand(residual_out, "residual_out", _F16, shape, dev)
    M = x.numel() // K if K else 0
    if (M | K) >> 31:
        M, K = _int32(M, K)
    _check(lib().qlinear_rms_norm(xp, rp, wp, M, K, eps, op, hp, _stream(dev)), "qlinear_rms_norm")
    return out


# ---------------------------------------------------------------- log probabilities

MAX_TOP = 64


class TokenLogprobs(NamedTuple):
    """Results of token_logprobs; None where one was not asked for."""
    logprob: torch.Tensor | None          # float32 [rows]
    entropy: torch.Tensor | None          # float32 [rows]
    top_logprob: torch.Tensor | None      # float32 [rows][top]
    top_id: torch.Tensor | None           # int32 [rows][top]


def token_logprobs_workspace_bytes(rows: int, vocab: int, top: int = 0, dtype: torch.dtype = torch.float16) -> int:
    n = ctypes.c_size_t(0)
    sizes = _int32(int(rows), int(vocab), 8 * dtype.itemsize, int(top))
    _check(lib().qlinear_token_logprobs_workspace_bytes(*sizes, ctypes.byref(n)),
           "qlinear_token_logprobs_workspace_bytes")
    return int(n.value)


def token_logprobs_workspace(rows: int, vocab: int, top: int = 0, dtype: torch.dtype = torch.float16,
                             device="cuda") -> torch.Tensor:
    """A token_logprobs workspace for calls of up to these sizes with logits of
    this type (scratch: needs no initialization; calls that may overlap in time
    must not share one)."""
    n = token_logprobs_workspace_bytes(rows, vocab, top, dtype)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, top: int = 0, entropy: bool = True,
                   out: TokenLogprobs | None = None, workspace: torch.Tensor | None = None) -> TokenLogprobs:
    """What rows of logits say (natural logarithms): the log probabilities of
    the given tokens (int32 [rows]), the entropies, and the `top` likeliest
    tokens with their log probabilities, largest first, equal ones by index.

    logits float16 or float32 [rows][vocab], row stride free. A row that holds
    +infinity or NaN, or -infinity alone, has NaN for log probabilities and
    entropy, and so has a token outside the vocabulary. out: a result of a call
    with the same rows, top, tokens and entropy, written again.
    """
    dev = _gpu_of(logits, "logits")
    if _current_gpu() != dev:
        with torch.cuda.device(dev):
            return token_logprobs(logits, tokens, top, entropy, out, workspace)
    if logits.dim() != 2 or (logits.dtype is not _F16 and logits.dtype is not _F32):
        raise ValueError(f"logits must be float16 or float32 [rows][vocab], got {logits.dtype} {tuple(logits.shape)}")
    R, V = logits.shape
    stride, along = logits.stride()
    if V > 1 and along != 1:
        raise ValueError("logits: the elements of a row must be contiguous")
    if R < 2:
        stride = V
    bits = 16 if logits.dtype is _F16 else 32
    tp = None if tokens is None else _operand(tokens, "tokens", _I32, (R,), dev)
    lp = ep = vp = ip = None
    if out is None:
        on = logits.device
        logprob = h = values = ids = None
        if tp is not None:
            logprob = torch.empty(R, dtype=_F32, device=on)
            lp = logprob.data_ptr()
        if entropy:
            h = torch.empty(R, dtype=_F32, device=on)
            ep = h.data_ptr()
        if top > 0:
            values, ids = torch.empty((R, top), dtype=_F32, device=on), torch.empty((R, top), dtype=_I32, device=on)
            vp, ip = values.data_ptr(), ids.data_ptr()
        out = TokenLogprobs(logprob, h, values, ids)
    else:
        wanted = (tokens is not None, bool(entropy), top > 0, top > 0)
        if any(w != (t is not None) for w, t in zip(wanted, out)):
            raise ValueError("out must hold what is asked for and None for the rest")
        if tokens is not None:
            lp = _operand(out.logprob, "logprob", _F32, (R,), dev)
        if entropy:
            ep = _operand(out.entropy, "entropy", _F32, (R,), dev)
        if top > 0:
            vp = _operand(out.top_logprob, "top_logprob", _F32, (R, top), dev)
            ip = _operand(out.top_id, "top_id", _I32, (R, top), dev)
    if (R | V | top) >> 31:
        R, V, top = _int32(R, V, top)
    n = ctypes.c_size_t(0)
    if workspace is None:
        _check(lib().qlinear_token_logprobs_workspace_bytes(R, V, bits, top, ctypes.byref(n)),
               "qlinear_token_logprobs_workspace_bytes")
        if n.value:
            workspace = torch.empty(n.value, dtype=_U8, device=logits.device)
    size = 0 if workspace is None else workspace.numel()
    wp = None if workspace is None else _operand(workspace, "workspace", _U8, (size,), dev)
    _check(lib().qlinear_token_logprobs(logits.data_ptr(), stride, R, V, bits, tp, top, lp, ep, vp, ip, wp, size,
                                        _stream(dev)), "qlinear_token_logprobs")
    return out
