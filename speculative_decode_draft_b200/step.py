"""The work around a speculative decode step's attention (include/wmtp_step.h).

PyTorch-facing wrappers in the manner of ``api.py``: encoded queries and keys in
the paged cache, page tables and slot maps on the device, log probabilities, and
the acceptance of drafted tokens.  Arguments are checked, outputs allocated and
the C calls made in ``csrc/step_binding.cpp``.

Every call runs on the device of its tensors, on ``stream`` or else on that
device's current stream; outputs and scratch that are not given are allocated
on that stream, so calls on several streams and in several captured graphs
share nothing.
"""

from __future__ import annotations

import ctypes
import importlib.util
import math
import os
from dataclasses import dataclass
from typing import Sequence

import torch

from . import _lib as L
from .api import I32, PagedCache

I64 = torch.int64
_CALLS = ("wmtp_qk_norm_rope", "wmtp_pages_resize", "wmtp_token_logprobs", "wmtp_accept_draft")
_native = None


def _binding():
    """The compiled binding, with the addresses of libwmtp's calls."""
    global _native
    if _native is None:
        lib = L.load()
        path = L.binding_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} not found; build it with `python -m speculative_decode_draft_b200.build` (needs "
                              "nvcc, a C++ compiler and the headers of Python and PyTorch)")
        spec = importlib.util.spec_from_file_location(f"{__package__}._step_binding", path)
        binding = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(binding)
        binding.init(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _CALLS))
        _native = binding
    return _native


def _on(stream, t) -> torch.cuda.StreamContext:
    """The context of ``stream``, which has to be on the device of ``t``."""
    if not isinstance(t, torch.Tensor) or stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {getattr(t, 'device', None)}")
    return torch.cuda.stream(stream)


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
    ``k_out`` is None unless given or the only place for the keys.  ``q_out`` may be ``q`` and ``k_out`` ``k``
    (contiguous, bf16); outputs that overlap q, k, v, one another or the pools otherwise are refused.
    """
    if stream is not None:
        with _on(stream, q if q is not None else k):
            return qk_norm_rope(p, rope, q, k, v, positions, slots=slots, cache=cache, q_weight=q_weight,
                                k_weight=k_weight, eps=eps, weight_offset=weight_offset, q_out=q_out, k_out=k_out,
                                status=status)
    turn, interleaved, factor = (None, False, 1.0) if rope is None else (rope.turn, rope.interleaved, rope.factor)
    k_pool, v_pool = (None, None) if cache is None else (cache.k_pool, cache.v_pool)
    code, q_out, k_out = (_native or _binding()).qk_norm_rope(
        p, turn, interleaved, factor, q, k, v, positions, slots, k_pool, v_pool, q_weight, k_weight, eps, weight_offset,
        q_out, k_out, status)
    L.check("wmtp_qk_norm_rope", code)
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
    if stream is not None:
        with _on(stream, page_table):
            return pages_resize(p, pool, page_table, kv_len, new_len, max_tokens=max_tokens, status=status)
    code, cu, positions, slots = (_native or _binding()).pages_resize(p, pool.free, pool.count, page_table, kv_len,
                                                                      new_len, max_tokens, status)
    L.check("wmtp_pages_resize", code)
    return None if cu is None else SlotMap(cu, positions, slots)


# ---------------------------------------------------------------- logits
@dataclass
class TokenLogprobs:
    logprobs: torch.Tensor             # [rows, num_tokens] fp32
    entropy: torch.Tensor              # [rows] fp32
    lse: torch.Tensor                  # [rows] fp32
    top_logprobs: torch.Tensor | None  # [rows, top_k] fp32
    top_ids: torch.Tensor | None       # [rows, top_k] int32


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, *, top_k: int = 0,
                   temperature: torch.Tensor | None = None, status=None, stream=None) -> TokenLogprobs:
    """Log probabilities of ``tokens`` int32 ``[rows, n]`` under ``logits [rows, vocab]``, each row's entropy and
    log-sum-exp, and its ``top_k`` (up to 64) most likely tokens (``wmtp_token_logprobs``).

    ``logits``: bf16, fp16 or fp32, rows ``vocab`` elements apart or more.  ``temperature`` fp32 ``[rows]``, above 0
    (at least 4.25e-39).
    """
    if stream is not None:
        with _on(stream, logits):
            return token_logprobs(logits, tokens, top_k=top_k, temperature=temperature, status=status)
    code, *out = (_native or _binding()).token_logprobs(logits, tokens, top_k, temperature, status)
    L.check("wmtp_token_logprobs", code)
    return TokenLogprobs(*out)


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
    were drafted, at most gamma.  ``temperature`` fp32 ``[B]``, at least 4.25e-39; 0 is
    greedy.
    """
    if stream is not None:
        with _on(stream, target_logits):
            return accept_draft(target_logits, draft_tokens, uniforms, draft_logits=draft_logits, num_draft=num_draft,
                                temperature=temperature, status=status)
    code, *out = (_native or _binding()).accept_draft(target_logits, draft_tokens, uniforms, draft_logits, num_draft,
                                                      temperature, status)
    L.check("wmtp_accept_draft", code)
    return Accepted(*out)
