"""The work around a speculative decode step's attention (include/wmtp_step.h).

PyTorch-facing wrappers, argument marshalling only, in the manner of
``api.py``: encoded queries and keys in the paged cache, page tables and slot
maps on the device, log probabilities, and the acceptance of drafted tokens.

Every call runs on the device of its tensors, on ``stream`` or else on that
device's current stream; outputs and scratch that are not given are allocated
on that stream, so calls on several streams and in several captured graphs
share nothing.
"""

from __future__ import annotations

import functools
import math
from ctypes import byref, c_size_t
from dataclasses import dataclass
from typing import Sequence

import torch

from . import _lib as L
from .api import BF16, I32, PagedCache, _need, _ptr, params

F32 = torch.float32
I64 = torch.int64
_DTYPES = {BF16: L.DTYPE_BF16, torch.float16: L.DTYPE_FP16, F32: L.DTYPE_FP32}


# torch.cuda.current_stream(i).cuda_stream without the Stream object, where there is such a call
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda i: torch.cuda.current_stream(i).cuda_stream)


def _elsewhere(index: int, stream):
    """The context that makes device ``index`` and ``stream`` current, None where they are."""
    if stream is None:
        return None if index == torch.cuda.current_device() else torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{index}")
    return torch.cuda.stream(stream)


def _cuda(t: torch.Tensor, name: str) -> int:
    """The tensor's device index."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _shaped(t: torch.Tensor, dtype, name: str, index: int, shape) -> None:
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        return
    _need(t, dtype, name, torch.device("cuda", index))  # says what is wrong
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _check_status(status, index: int) -> None:
    if status is not None:
        _need(status, I32, "status", torch.device("cuda", index))


# ---------------------------------------------------------------- rotary positions
def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str = "none", stretch: float = 1.0,
                     original: int = 0, fast: float = 32.0, slow: float = 1.0) -> list[float]:
    """Angle per position of each pair, ``base ** (-2 i / rotary_dim)``, scaled for long contexts.

    ``scaling``: ``"none"``; ``"linear"`` divides every angle by ``stretch``; the two others divide only the
    angles of pairs that turn rarely in ``original`` positions and leave fast ones as they are, with a ramp
    between: ``"bands"`` by the turns themselves (kept from ``fast`` turns on, divided up to ``slow``),
    ``"yarn"`` by the pair's index (from the pair that makes ``fast`` turns to the one that makes ``slow``,
    rounded outwards).
    """
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    freq = [float(base) ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if scaling == "none":
        return freq
    if not stretch > 0.0:
        raise ValueError("stretch must be positive")
    if scaling == "linear":
        return [f / stretch for f in freq]
    if scaling not in ("yarn", "bands"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if original <= 0 or not fast > slow > 0.0:
        raise ValueError(f"{scaling} needs original > 0 and fast > slow > 0")
    if scaling == "bands":
        keep = [min(max((original * f / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0) for f in freq]
    else:
        def pair(turns: float) -> float:
            return rotary_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rotary_dim - 1)
        keep = [1.0 - min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(rotary_dim // 2)]
    return [f * k + f / stretch * (1.0 - k) for f, k in zip(freq, keep)]


@dataclass
class Rope:
    """Rotary positions of ``qk_norm_rope`` (``wmtp_rope``).

    ``turn`` int64 ``[rotary_dim / 2]`` (device): each pair's turns per position, in units of 2^-64 turn.
    ``factor`` multiplies the rotated elements.
    """
    turn: torch.Tensor
    interleaved: bool = False
    factor: float = 1.0

    @staticmethod
    def from_frequencies(freq: Sequence[float], *, interleaved: bool = False, factor: float = 1.0,
                         device="cuda") -> "Rope":
        """From each pair's angle per position in radians (``rope_frequencies``, say)."""
        turn = []
        for f in freq:
            if not math.isfinite(f):
                raise ValueError("frequencies must be finite")
            t = int(float(f) / (2 * math.pi) * 2.0 ** 64) % (1 << 64)
            turn.append(t - (1 << 64) if t >> 63 else t)  # as int64 bits
        return Rope(torch.tensor(turn, dtype=I64, device=device), interleaved, float(factor))

    def desc(self) -> L.RopeDesc:
        _need(self.turn, I64, "turn")
        return L.RopeDesc(self.turn.data_ptr(), 2 * self.turn.numel(), int(bool(self.interleaved)), self.factor)


def _heads(t: torch.Tensor, name: str, index: int, dtype, lead, heads: int, dim: int):
    """(pointer, token stride, head stride) of a ``[..., heads, dim]`` view with one token stride."""
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (*lead, heads, dim):
        raise ValueError(f"{name} must be {[*lead, heads, dim]}, got {list(t.shape)}")
    st = t.stride()
    if dim > 1 and st[-1] != 1:
        raise ValueError(f"{name}: the elements of a head must be next to one another")
    token = st[0]  # strides of axes with one entry say nothing
    if len(lead) == 1:
        if lead[0] <= 1:
            token = 0
    elif lead[1] > 1:
        if lead[0] > 1 and st[0] != lead[1] * st[1]:
            raise ValueError(f"{name}: tokens must be evenly spaced")
        token = st[1]
    elif lead[0] <= 1:
        token = 0
    return t.data_ptr(), token, st[-2] if heads > 1 else 0


def qk_norm_rope(p: L.Params, rope: Rope | None, q: torch.Tensor | None, k: torch.Tensor | None,
                 v: torch.Tensor | None, positions: torch.Tensor, *, slots: torch.Tensor | None = None,
                 cache: PagedCache | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, weight_offset: float = 0.0, q_out=None,
                 k_out=None, status=None, stream=None):
    """Encode a step's queries and keys, and write K and V into the paged cache -> (q_out, k_out).

    Per head: RMS norm (where a weight is given), then the position rotation, in fp32, rounded to bf16 once
    (``wmtp_qk_norm_rope``).  ``q [T, Hq, D]`` or ``[B, n, Hq, D]``, ``k``, ``v`` likewise with ``Hkv``: bf16
    or fp32, views cut from one packed projection too.  ``positions`` int32, one per token; a token with a
    negative position is padding and leaves everything as it was.  ``slots`` int64, one per token: where K and V
    go in ``cache``'s pools (``pages_resize`` makes both).  Without slots the keys are returned only (``v`` None).
    ``k_out`` is None unless given or the only place for the keys.
    """
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k is needed")
    dev = _cuda(first, "q" if q is not None else "k")
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return qk_norm_rope(p, rope, q, k, v, positions, slots=slots, cache=cache, q_weight=q_weight,
                                k_weight=k_weight, eps=eps, weight_offset=weight_offset, q_out=q_out, k_out=k_out,
                                status=status)
    dt = first.dtype
    if dt is not BF16 and dt is not F32:
        raise TypeError(f"q, k and v must be bf16 or fp32, got {dt}")
    if first.dim() not in (3, 4):
        raise ValueError("q and k must be [tokens, heads, dim] or [batch, tokens, heads, dim]")
    lead = tuple(first.shape[:-2])
    Hq, Hkv, D = p.num_heads_q, p.num_heads_kv, p.head_dim
    tokens = math.prod(lead)
    none = (None, 0, 0)
    qa = none if q is None else _heads(q, "q", dev, dt, lead, Hq, D)
    ka = none if k is None else _heads(k, "k", dev, dt, lead, Hkv, D)
    va = none if v is None else _heads(v, "v", dev, dt, lead, Hkv, D)
    _shaped(positions, I32, "positions", dev, lead)
    kv = None
    if slots is not None:
        _shaped(slots, I64, "slots", dev, lead)
        if cache is None:
            raise ValueError("slots need a cache")
        kp, vp = cache.k_pool, cache.v_pool
        pool = (kp.shape[0], Hkv, p.page_size, D)
        _shaped(kp, BF16, "cache.k_pool", dev, pool)
        _shaped(vp, BF16, "cache.v_pool", dev, pool)
        kv = byref(L.PagedKVDesc(kp.data_ptr(), vp.data_ptr(), pool[0], None, 0, None))
    wt = BF16
    for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            wt = w.dtype
            if wt is not BF16 and wt is not F32:
                raise TypeError(f"{n} must be bf16 or fp32")
            _shaped(w, wt, n, dev, (D,))
    if q_weight is not None and k_weight is not None and q_weight.dtype is not k_weight.dtype:
        raise TypeError("q_weight and k_weight must have one dtype")
    rd = None
    if rope is not None:
        if rope.turn.get_device() != dev:
            raise ValueError(f"rope is on {rope.turn.device}, expected cuda:{dev}")
        rd = byref(rope.desc())
    if q_out is not None:
        _shaped(q_out, BF16, "q_out", dev, (*lead, Hq, D))
    elif q is not None:
        q_out = torch.empty(q.shape, dtype=BF16, device=q.device)
    if k_out is not None:
        _shaped(k_out, BF16, "k_out", dev, (*lead, Hkv, D))
    elif k is not None and slots is None:
        k_out = torch.empty(k.shape, dtype=BF16, device=k.device)
    _check_status(status, dev)
    if tokens:  # empty tensors have no address
        L.check("wmtp_qk_norm_rope", L.load().wmtp_qk_norm_rope(
            byref(p), rd, tokens, _DTYPES[dt], *qa, *ka, *va, positions.data_ptr(), _ptr(slots), kv, _ptr(q_weight),
            _ptr(k_weight), _DTYPES[wt], weight_offset, eps, _ptr(q_out), _ptr(k_out), _ptr(status),
            _current_stream(dev)))
    return q_out, k_out


# ---------------------------------------------------------------- pages
@dataclass
class DevicePages:
    """The free pages of one pool, in device memory: a stack of page indices.

    ``free`` int32 ``[num_pages]``, the first ``count[0]`` entries are free; ``count`` int32 ``[1]``.
    """
    free: torch.Tensor
    count: torch.Tensor

    @staticmethod
    def allocate(num_pages: int, device="cuda") -> "DevicePages":
        """All of ``num_pages`` free; page 0 is taken first."""
        return DevicePages(torch.arange(num_pages - 1, -1, -1, dtype=I32, device=device),
                           torch.full((1,), num_pages, dtype=I32, device=device))


@dataclass
class SlotMap:
    """Where the tokens that ``pages_resize`` added go.

    Sequence b's are rows ``cu_tokens[b]`` to ``cu_tokens[b + 1]``; rows behind the last one hold -1.
    """
    cu_tokens: torch.Tensor  # [B + 1] int32
    positions: torch.Tensor  # [max_tokens] int32
    slots: torch.Tensor      # [max_tokens] int64


def pages_resize(p: L.Params, pool: DevicePages, page_table: torch.Tensor, kv_len: torch.Tensor,
                 new_len: torch.Tensor, *, max_tokens: int = 0, status=None, stream=None) -> SlotMap | None:
    """Take every sequence from ``kv_len`` to ``new_len`` tokens (``wmtp_pages_resize``).

    ``page_table`` int32 ``[B, max_pages]``, ``kv_len`` int32 ``[B]`` and the pool are updated in place: pages
    above the new length go back, missing ones are taken.  With ``max_tokens`` the added tokens' positions and
    cache slots are returned, as ``qk_norm_rope`` takes them.
    """
    dev = _cuda(page_table, "page_table")
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return pages_resize(p, pool, page_table, kv_len, new_len, max_tokens=max_tokens, status=status)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    B, width = page_table.shape
    _shaped(page_table, I32, "page_table", dev, (B, width))
    _shaped(kv_len, I32, "kv_len", dev, (B,))
    _shaped(new_len, I32, "new_len", dev, (B,))
    pages = pool.free.numel()
    _shaped(pool.free, I32, "pool.free", dev, (pages,))
    _shaped(pool.count, I32, "pool.count", dev, (1,))
    _check_status(status, dev)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    device = page_table.device
    out, ptrs = None, (None, None, None)
    if max_tokens:
        out = SlotMap(torch.empty(B + 1, dtype=I32, device=device), torch.empty(max_tokens, dtype=I32, device=device),
                      torch.empty(max_tokens, dtype=I64, device=device))
        ptrs = (out.cu_tokens.data_ptr(), out.positions.data_ptr(), out.slots.data_ptr())
    nbytes = _pages_bytes(p.page_size, B, width, pages, max_tokens)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    L.check("wmtp_pages_resize", L.load().wmtp_pages_resize(
        byref(p), B, page_table.data_ptr(), width, kv_len.data_ptr(), new_len.data_ptr(), pool.free.data_ptr(),
        pool.count.data_ptr(), pages, *ptrs, max_tokens, _ptr(ws), byref(c_size_t(nbytes)), _ptr(status),
        _current_stream(dev)))
    return out


@functools.lru_cache(maxsize=256)
def _pages_bytes(page_size: int, batch: int, width: int, pages: int, max_tokens: int) -> int:
    """Scratch of a call of these sizes (the head counts do not matter)."""
    size = c_size_t(0)
    anything = 256 if max_tokens else None  # never read: a size query
    L.check("wmtp_pages_resize", L.load().wmtp_pages_resize(
        byref(params(1, 1, 64, page_size=page_size)), batch, None, width, None, None, None, None, pages, anything,
        anything, anything, max_tokens, None, byref(size), None, None))
    return size.value


# ---------------------------------------------------------------- logits
@dataclass
class TokenLogprobs:
    logprobs: torch.Tensor             # [rows, num_tokens] fp32
    entropy: torch.Tensor              # [rows] fp32
    lse: torch.Tensor                  # [rows] fp32
    top_logprobs: torch.Tensor | None  # [rows, top_k] fp32
    top_ids: torch.Tensor | None       # [rows, top_k] int32


def _row_stride(t: torch.Tensor, axis: int) -> int:
    return t.stride(axis) if t.shape[axis] > 1 else t.shape[-1]


def _logits_ok(t: torch.Tensor, name: str) -> None:
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be bf16, fp16 or fp32, got {t.dtype}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the logits of a row must be next to one another")


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, *, top_k: int = 0,
                   temperature: torch.Tensor | None = None, status=None, stream=None) -> TokenLogprobs:
    """Log probabilities of ``tokens`` int32 ``[rows, n]`` under ``logits [rows, vocab]``, each row's entropy and
    log-sum-exp, and its ``top_k`` (up to 64) most likely tokens (``wmtp_token_logprobs``).

    ``logits``: bf16, fp16 or fp32, rows any stride apart.  ``temperature`` fp32 ``[rows]``, above 0.
    """
    dev = _cuda(logits, "logits")
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return token_logprobs(logits, tokens, top_k=top_k, temperature=temperature, status=status)
    _logits_ok(logits, "logits")
    if logits.dim() != 2 or tokens.dim() != 2:
        raise ValueError("logits must be [rows, vocab] and tokens [rows, n]")
    R, V = logits.shape
    n = tokens.shape[1]
    _shaped(tokens, I32, "tokens", dev, (R, n))
    if temperature is not None:
        _shaped(temperature, F32, "temperature", dev, (R,))
    _check_status(status, dev)
    if top_k < 0:
        raise ValueError("top_k must not be negative")
    device = logits.device
    logprobs = torch.empty(R, n, dtype=F32, device=device)
    entropy = torch.empty(R, dtype=F32, device=device)
    lse = torch.empty_like(entropy)
    top_logprobs = top_ids = None
    if top_k:
        top_logprobs = torch.empty(R, top_k, dtype=F32, device=device)
        top_ids = torch.empty(R, top_k, dtype=I32, device=device)
    L.check("wmtp_token_logprobs", L.load().wmtp_token_logprobs(
        R, V, _DTYPES[logits.dtype], logits.data_ptr(), _row_stride(logits, 0), _ptr(temperature), tokens.data_ptr(),
        n, top_k, logprobs.data_ptr(), entropy.data_ptr(), lse.data_ptr(), _ptr(top_logprobs), _ptr(top_ids),
        _ptr(status), _current_stream(dev)))
    return TokenLogprobs(logprobs, entropy, lse, top_logprobs, top_ids)


@dataclass
class Accepted:
    tokens: torch.Tensor    # [B, num_q] int32: the emitted tokens, -1 behind them
    count: torch.Tensor     # [B] int32: how many
    logprobs: torch.Tensor  # [B, num_q] fp32: ln p of each under the target


def accept_draft(target_logits: torch.Tensor, draft_tokens: torch.Tensor, uniforms: torch.Tensor, *,
                 draft_logits: torch.Tensor | None = None, num_draft: torch.Tensor | None = None,
                 temperature: torch.Tensor | None = None, status=None, stream=None) -> Accepted:
    """Which drafted tokens the target accepts, and the token that follows them (``wmtp_accept_draft``).

    ``target_logits [B, gamma + 1, vocab]`` (a verify block's), ``draft_tokens`` int32 ``[B, gamma]``,
    ``uniforms`` fp32 ``[B, gamma + 1]`` in [0, 1).  ``draft_logits [B, gamma, vocab]``: the distributions that
    the tokens were drawn from; None if each was its draft's only choice.  ``num_draft`` int32 ``[B]``: how many
    were drafted, at most gamma.  ``temperature`` fp32 ``[B]``; 0 is greedy.
    """
    dev = _cuda(target_logits, "target_logits")
    away = _elsewhere(dev, stream)
    if away is not None:
        with away:
            return accept_draft(target_logits, draft_tokens, uniforms, draft_logits=draft_logits, num_draft=num_draft,
                                temperature=temperature, status=status)
    _logits_ok(target_logits, "target_logits")
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [batch, gamma + 1, vocab]")
    B, n, V = target_logits.shape
    if n < 1:
        raise ValueError("target_logits needs a row for the token that follows")
    _shaped(draft_tokens, I32, "draft_tokens", dev, (B, n - 1))
    _shaped(uniforms, F32, "uniforms", dev, (B, n))
    ds = (0, 0)
    if draft_logits is not None:
        _logits_ok(draft_logits, "draft_logits")
        if draft_logits.get_device() != dev or draft_logits.dtype is not target_logits.dtype:
            raise TypeError("draft_logits must have the device and dtype of target_logits")
        if draft_logits.shape != (B, n - 1, V):
            raise ValueError(f"draft_logits must be {[B, n - 1, V]}, got {list(draft_logits.shape)}")
        ds = (_row_stride(draft_logits, 0), _row_stride(draft_logits, 1))
    if num_draft is not None:
        _shaped(num_draft, I32, "num_draft", dev, (B,))
    if temperature is not None:
        _shaped(temperature, F32, "temperature", dev, (B,))
    _check_status(status, dev)
    device, dt = target_logits.device, _DTYPES[target_logits.dtype]
    nbytes = _accept_bytes(B, n, V, dt)
    ws = torch.empty(nbytes or 256, dtype=torch.uint8, device=device)
    tokens = torch.empty(B, n, dtype=I32, device=device)
    count = torch.empty(B, dtype=I32, device=device)
    logprobs = torch.empty_like(uniforms)
    L.check("wmtp_accept_draft", L.load().wmtp_accept_draft(
        B, n, V, dt, target_logits.data_ptr(), _row_stride(target_logits, 0), _row_stride(target_logits, 1),
        _ptr(draft_logits), *ds, draft_tokens.data_ptr(), uniforms.data_ptr(), _ptr(num_draft), _ptr(temperature),
        tokens.data_ptr(), count.data_ptr(), logprobs.data_ptr(), ws.data_ptr(), byref(c_size_t(nbytes or 256)),
        _ptr(status), _current_stream(dev)))
    return Accepted(tokens, count, logprobs)


@functools.lru_cache(maxsize=256)
def _accept_bytes(batch: int, num_q: int, vocab: int, dtype: int) -> int:
    """Scratch of a call of these sizes."""
    size = c_size_t(0)
    L.check("wmtp_accept_draft", L.load().wmtp_accept_draft(
        batch, num_q, vocab, dtype, None, 0, 0, None, 0, 0, None, None, None, None, None, None, None, None,
        byref(size), None, None))
    return size.value
