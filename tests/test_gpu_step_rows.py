"""token_logprobs and accept_draft of a row by itself and among others.

A row's sums are split over as many CTAs as its call has room for, so its bits depend on the number of rows; with the
same split they are the same.  Between two splits each value is off from the exact one by what test_gpu_step_logits.py
derives: for N columns and mean |y| E under the row's distribution a logarithm of the sum by
e = 2^-22 + (N / 256 + 40) 2^-24 + 4 * 2^-24 E, a log probability by that, 2 * 2^-24 ln S and 3 * 2^-24 |y|, the entropy by
(1 + E) e + 4 * 2^-24 E y^2 + 6 * 2^-24 (ln S + E).  Two of them differ by twice that; which tokens are largest does not
depend on the split at all.
"""

import numpy as np
import pytest
import torch

import speculative_decode_draft_b200 as w
from _helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
NAMES = ("logprobs", "entropy", "lse", "top_logprobs", "top_ids")


def _rows(seed, rows, vocab):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g, device=DEV) * 2).bfloat16()
    return x, torch.randint(0, vocab, (rows, 3), generator=g, device=DEV).int()


def _bounds(row):
    y = row - row.max()
    p = np.exp(y)
    s = p.sum()
    p /= s
    mean, square, ln = -(p * y).sum(), (p * y * y).sum(), np.log(s)
    e = 2.0 ** -22 + (len(row) / 256 + 40) * U + 4 * U * mean
    return y, 2 * (e + 2 * U * ln), 2 * (e + 2 * U * ln + 4 * U * (abs(row.max()) + ln)), 2 * ((1 + mean) * e + 4 * U * square
                                                                                          + 6 * U * (ln + mean))


def _compare(row, ids, a, b):
    """One row's results of two calls."""
    y, lp, lse, ent = _bounds(row)
    assert torch.equal(a["top_ids"], b["top_ids"])
    for name, at in (("logprobs", ids), ("top_logprobs", a["top_ids"].tolist())):
        for u, v, j in zip(f64(a[name]), f64(b[name]), at):
            assert abs(u - v) <= lp + 6 * U * abs(y[j])
    assert abs(float(a["lse"]) - float(b["lse"])) <= lse and abs(float(a["entropy"]) - float(b["entropy"])) <= ent


@pytest.mark.parametrize("rows,vocab", [(2, 40000), (9, 40000), (150, 5001), (300, 40000), (700, 30001)])
def test_logprobs_of_a_row_alone_and_in_a_batch(cuda_device, rows, vocab):
    x, ids = _rows(rows, rows, vocab)
    whole = w.token_logprobs(x, ids, top_k=9)
    for i in sorted({0, 1, rows // 2, rows - 1}):
        one = w.token_logprobs(x[i:i + 1], ids[i:i + 1], top_k=9)
        _compare(f64(x[i]), ids[i].tolist(), {n: getattr(one, n)[0] for n in NAMES}, {n: getattr(whole, n)[i] for n in NAMES})


def test_logprobs_have_the_same_bits_where_rows_are_split_alike(cuda_device):
    """1 to 64 rows of 40000: as many CTAs a row as there may be; 700 and 1000: one."""
    for few, many in ((1, 64), (7, 64), (700, 1000)):
        x, ids = _rows(many, many, 40000)
        a, b = w.token_logprobs(x[:few], ids[:few], top_k=9), w.token_logprobs(x, ids, top_k=9)
        for n in NAMES:
            assert torch.equal(getattr(a, n), getattr(b, n)[:few]), (few, many, n)


def test_acceptance_of_a_sequence_alone_and_in_a_batch(cuda_device):
    """Which drafts are accepted and what is drawn; uniforms are kept clear of the borders by the drafts' choice: the
    likeliest token with u = 0.001, and one of nearly no probability with u = 0.9."""
    B, G, V = 300, 3, 20000
    x, _ = _rows(7, B * (G + 1), V)
    x = x.view(B, G + 1, V)
    best, worst = x[:, :G].float().argmax(-1).int(), x[:, :G].float().argmin(-1).int()
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    likely = torch.rand(B, G, generator=g, device=DEV) < 0.7
    x[:, :G].scatter_add_(-1, best.long()[..., None], torch.full((B, G, 1), 12.0, device=DEV).bfloat16())
    drafts = torch.where(likely, best, worst)
    u = torch.full((B, G + 1), 0.5, device=DEV)
    u[:, :G] = torch.where(likely, 0.001, 0.9)
    whole = w.accept_draft(x, drafts, u)
    expect = likely.int().cumprod(1).sum(1) + 1
    assert torch.equal(whole.count, expect.int())
    for i in (0, 1, 150, 299):
        one = w.accept_draft(x[i:i + 1], drafts[i:i + 1], u[i:i + 1])
        n = int(expect[i])
        assert torch.equal(one.count, whole.count[i:i + 1])
        assert torch.equal(one.tokens[0, :n - 1], whole.tokens[i, :n - 1])  # the drafts; the draw's border has bits of its own
        same = one.tokens[0] == whole.tokens[i]
        for j in range(n):
            if same[j]:
                y, lp, _, _ = _bounds(f64(x[i, j]))
                assert abs(float(one.logprobs[0, j]) - float(whole.logprobs[i, j])) <= lp + 6 * U * abs(y[int(one.tokens[0, j])])
