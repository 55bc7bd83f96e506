"""Plain fp64 versions of the work around the attention (include/wmtp_step.h):
norm and rotation of heads, page tables, log probabilities, acceptance.

One token, page, row or sequence at a time, straight from the formulas.
"""

from __future__ import annotations

import math

import numpy as np


def rotate_heads(x, positions, freq, *, interleaved=False, factor=1.0, weight=None, offset=0.0, eps=1e-6):
    """``x [T, H, D]`` -> the normed (``weight [D]`` given) and rotated heads.

    ``freq``: angle per position of each pair.  The angles are taken in 80
    bits: 64 lose 1e-7 of one at position 2^31.
    """
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + offset)
    n = len(freq)
    first = np.arange(n) * 2 if interleaved else np.arange(n)
    second = first + 1 if interleaved else first + n
    angle = np.asarray(positions).astype(np.longdouble)[:, None, None] * np.asarray(freq, np.float64).astype(
        np.longdouble)
    cos, sin = (np.asarray(f(angle), np.float64) * factor for f in (np.cos, np.sin))
    a, b = y[..., first].copy(), y[..., second].copy()
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


class PageModel:
    """Page tables, lengths and the free stack of one pool, as Python lists."""

    def __init__(self, page_size, num_pages, table, kv_len, free):
        self.P, self.num_pages = page_size, num_pages
        self.table = [list(map(int, r)) for r in table]
        self.kv_len = list(map(int, kv_len))
        self.free = list(map(int, free))

    def resize(self, new_len, max_tokens=0):
        """-> (cu, positions, slots, what went wrong as a set of names)."""
        P, cap, wrong = self.P, len(self.table[0]) * self.P if self.table else 0, set()
        ok = []
        for b, (old, new) in enumerate(zip(self.kv_len, new_len)):
            ok.append(0 <= old <= cap and 0 <= new <= cap)
            if not ok[b]:
                wrong.add("len")
        give = []
        for b, new in enumerate(new_len):
            if ok[b]:
                give += [(b, j) for j in range(-(-int(new) // P), -(-self.kv_len[b] // P))]
        cu, positions, slots = [0], [], []
        if len(self.free) + len(give) > self.num_pages:
            cu = [0] * (len(self.table) + 1)
            return cu, [-1] * max_tokens, [-1] * max_tokens, wrong | {"pool"}
        for b, j in reversed(give):  # highest first
            self.free.append(self.table[b][j])
            self.table[b][j] = -1
        stopped = False
        for b, new in enumerate(map(int, new_len)):
            old = self.kv_len[b]
            grow = new - old
            if ok[b] and grow > 0:
                need = -(-new // P) - -(-old // P)
                stopped = stopped or need > len(self.free) or (max_tokens and len(slots) + grow > max_tokens)
                if stopped:
                    wrong.add("pool")
                else:
                    for j in range(-(-old // P), -(-new // P)):
                        self.table[b][j] = self.free.pop()
                    if max_tokens:
                        for t in range(old, new):
                            page = self.table[b][t // P]
                            positions.append(t)
                            slots.append(page * P + t % P if 0 <= page < self.num_pages else -1)
                            if slots[-1] < 0:
                                wrong.add("page")
                    self.kv_len[b] = new
            elif ok[b]:
                self.kv_len[b] = new
            cu.append(len(slots))
        behind = [-1] * (max_tokens - len(slots))
        return cu, positions + behind, slots + behind, wrong


def row_logprobs(row, temperature=1.0):
    """(log probabilities, lse, entropy) of one row of logits."""
    y = np.asarray(row, np.float64) / temperature
    m = y.max()
    if m == -math.inf:
        return np.full_like(y, -math.inf), -math.inf, 0.0
    lse = m + math.log(np.exp(y - m).sum())
    lp = y - lse
    there = np.isfinite(lp)
    return lp, lse, float(-(np.exp(lp[there]) * lp[there]).sum())


def top_tokens(row, k):
    """The k largest logits' ids: larger first, equal ones by lower id, masked ones never; -1 behind them."""
    row = np.asarray(row, np.float64)
    ids = [int(i) for i in np.lexsort((np.arange(len(row)), -row))[:k] if row[i] > -math.inf]
    return ids + [-1] * (k - len(ids))


def accept_sequence(target, draft_tokens, uniforms, draft=None, num_draft=None, temperature=1.0):
    """One sequence -> (emitted tokens, their log probabilities, margin).

    ``target [n, V]``, ``draft [n - 1, V]`` or None (all weight on the drafted
    token).  ``margin``: how far, relative to what was compared, the nearest
    decision was from going the other way.
    """
    target = np.asarray(target, np.float64)
    n = len(target)
    nd = n - 1 if num_draft is None else num_draft
    t = temperature if temperature > 0 else 1.0
    tokens, logps, margin, k, rejected = [], [], math.inf, 0, False
    while k < nd:
        d = int(draft_tokens[k])
        lp, _, _ = row_logprobs(target[k], t)
        if temperature == 0:
            ok = d == int(np.argmax(target[k]))
        elif 0 <= d < target.shape[1]:
            q = 1.0 if draft is None else math.exp(row_logprobs(draft[k], t)[0][d])
            p, uq = math.exp(lp[d]), float(uniforms[k]) * q
            ok = uq < p
            margin = min(margin, abs(uq - p) / max(uq, p)) if max(uq, p) > 0 else margin
        else:
            ok = False
        if not ok:
            rejected = True
            break
        tokens.append(d)
        logps.append(lp[d])
        k += 1
    lp, _, _ = row_logprobs(target[k], t)
    if temperature == 0:
        pick = int(np.argmax(target[k]))
    else:
        p = np.exp(lp)
        w = p
        if rejected:
            d = int(draft_tokens[k])
            if draft is None:
                w = p.copy()
                if 0 <= d < len(p):
                    w[d] = 0.0
            else:
                w = np.maximum(p - np.exp(row_logprobs(draft[k], t)[0]), 0.0)
            if not w.sum() > 0:
                w = p
        mass = np.cumsum(w)
        want = float(uniforms[n - 1]) * mass[-1]
        pick = int(np.argmax(mass > want))
        below = mass[pick - 1] if pick else 0.0
        margin = min(margin, (mass[pick] - want) / mass[-1] * 1e3, (want - below) / mass[-1] * 1e3 if pick else math.inf)
    return tokens + [pick], logps + [lp[pick]], margin
