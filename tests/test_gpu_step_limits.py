"""token_logprobs and accept_draft at the ends of the temperatures' range.

At a temperature T of 1e28 and above every finite logit of ordinary size has the same weight; a masked one has
none at any temperature.  Where one token is left its log probability is exactly 0, as ln 1 and 0 / T are.

Above 2^126 the reciprocal of T is subnormal: 1 / T >= 2^-128 is off by 2^-150, a relative 2^-22, and log2(e) / T by
as much again.  With |y| <= 2 the exponents y log2(e) are below 3 and off by 3 (2 * 2^-22 + 2 * 2^-24), each term of a
row's sum then by ln 2 times that and the 2^-22 of the hardware's 2^x, together below 2^-19, as the sum, its
logarithm and the y (2 * 2^-22) beside it; 2^-18 for a difference of both.
"""

import numpy as np
import pytest
import torch

import oracle
import speculative_decode_draft_b200 as w
from speculative_decode_draft_b200 import _lib as L
from _helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NEG = float("-inf")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HIGH = [1e20, 1e28, 1e29, 1e30, 1e35, 1e38, 3e38]


def _temps(rows, t):
    return torch.full((rows,), t, device=DEV)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 7), (4, 5001), (2, 131072), (700, 1500)])
@pytest.mark.parametrize("t", HIGH)
def test_rows_of_masked_tokens_alone_at_high_temperatures(cuda_device, dtype, rows, vocab, t):
    x = torch.full((rows, vocab), NEG, dtype=DT[dtype], device=DEV)
    ids = torch.zeros(rows, 1, dtype=torch.int32, device=DEV)
    status = w.new_status(DEV)
    r = w.token_logprobs(x, ids, top_k=2, temperature=_temps(rows, t), status=status)
    assert int(status.item()) == 0
    assert (r.lse == NEG).all() and (r.entropy == 0).all() and (r.logprobs == NEG).all()
    assert (r.top_ids == -1).all() and (r.top_logprobs == NEG).all()
    none = torch.zeros(rows, 0, dtype=torch.int32, device=DEV)
    a = w.accept_draft(x[:, None], none, torch.full((rows, 1), 0.5, device=DEV), temperature=_temps(rows, t), status=status)
    assert int(status.item()) == L.DEV_LOGITS
    assert (a.count == 0).all() and (a.tokens == -1).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,vocab", [(3, 7), (4, 5001), (2, 131072), (700, 1500)])
@pytest.mark.parametrize("t", HIGH)
@pytest.mark.parametrize("where", ["first", "last"])
def test_one_token_left_at_high_temperatures(cuda_device, dtype, rows, vocab, t, where):
    at = 0 if where == "first" else vocab - 1
    x = torch.full((rows, vocab), NEG, dtype=DT[dtype], device=DEV)
    x[:, at] = 1.0
    ids = torch.tensor([[at, vocab // 2]] * rows, dtype=torch.int32, device=DEV)
    status = w.new_status(DEV)
    r = w.token_logprobs(x, ids, top_k=2, temperature=_temps(rows, t), status=status)
    assert (r.logprobs[:, 0] == 0).all() and (r.logprobs[:, 1] == NEG).all() and (r.entropy == 0).all()
    assert (r.lse.double() - 1 / t).abs().max() <= 2.0 ** -149 + 2.0 ** -22 / t
    assert (r.top_ids == torch.tensor([at, -1], device=DEV)).all() and (r.top_logprobs[:, 0] == 0).all()
    drafts = torch.full((rows, 1), vocab // 2, dtype=torch.int32, device=DEV)
    drafts[::2] = at
    a = w.accept_draft(x[:, None].expand(rows, 2, vocab), drafts, torch.full((rows, 2), 0.9, device=DEV),
                       temperature=_temps(rows, t), status=status)
    assert int(status.item()) == 0
    assert (a.count[::2] == 2).all() and (a.tokens[::2] == at).all() and (a.logprobs == 0).all()
    assert (a.count[1::2] == 1).all() and (a.tokens[1::2] == torch.tensor([at, -1], device=DEV)).all()


@pytest.mark.parametrize("t", [1e38, 3e38])
@pytest.mark.parametrize("vocab", [9, 5001, 131072])
def test_few_tokens_left_of_the_size_of_a_high_temperature(cuda_device, t, vocab):
    """The live logits lie in one thread's columns; every other thread and CTA has masked ones alone."""
    x = torch.full((2, vocab), NEG, device=DEV)
    x[:, 1:4] = torch.tensor([-t, 0.0, t / 2], device=DEV)
    ids = torch.tensor([[1, 2, 3]] * 2, dtype=torch.int32, device=DEV)
    temps = _temps(2, t)
    r = w.token_logprobs(x, ids, temperature=temps)
    for i in range(2):
        ref, lse, ent = oracle.row_logprobs(f64(x[i]), float(temps[i]))
        assert np.abs(f64(r.logprobs[i]) - ref[1:4]).max() <= 2.0 ** -18
        assert abs(float(r.lse[i]) - lse) <= 2.0 ** -18 and abs(float(r.entropy[i]) - ent) <= 2.0 ** -17


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [4, 5001, 131072])
@pytest.mark.parametrize("t", [2.0, 64.0, 1e10])
def test_differences_of_logits_beyond_fp32(cuda_device, dtype, vocab, t):
    """x - max passes fp32, (x - max) / T does not: the log probability is finite, off by the roundings of 1 / T, the
    difference and the product."""
    x = torch.full((2, vocab), NEG, device=DEV)
    x[:, 0], x[:, -1], x[1, 1] = 3e38, -3e38, -2e38
    x = x.to(DT[dtype])
    ids = torch.tensor([[0, vocab - 1, 1]] * 2, dtype=torch.int32, device=DEV)
    r = w.token_logprobs(x, ids, top_k=3, temperature=_temps(2, t))
    want = (f64(x) - f64(x).max(-1, keepdims=True)) / f64(_temps(2, t))[:, None]
    for i in range(2):
        for got, j in zip(f64(r.logprobs[i]), ids[i].tolist()):
            assert got == want[i, j] or abs(got - want[i, j]) <= 3 * 2.0 ** -24 * abs(want[i, j]), (i, j, got)
        ranked = oracle.top_tokens(f64(x[i]), 3)
        assert r.top_ids[i].tolist() == ranked and (r.entropy == 0).all()
        for got, j in zip(f64(r.top_logprobs[i]), ranked):
            assert got == (want[i, j] if j >= 0 else NEG) or abs(got - want[i, j]) <= 3 * 2.0 ** -24 * abs(want[i, j])


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("t", [1e38, 3e38])
def test_acceptance_of_logits_of_the_size_of_a_high_temperature(cuda_device, t, drafted):
    B, V = 200, 5001
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.full((B, 2, V), NEG, device=DEV)
    x[..., 1:4] = torch.tensor([-t, 0.0, t / 2], device=DEV)
    q = torch.full((B, 1, V), NEG, device=DEV)
    q[..., 1:4] = torch.tensor([t / 2, -t, 0.0], device=DEV)
    tokens = torch.randint(1, 4, (B, 1), generator=g, device=DEV).int()
    u = torch.rand(B, 2, generator=g, device=DEV)
    status = w.new_status(DEV)
    r = w.accept_draft(x, tokens, u, draft_logits=q if drafted else None, temperature=_temps(B, t), status=status)
    assert int(status.item()) == 0
    clear = 0
    for b in range(B):
        ids, logps, margin = oracle.accept_sequence(f64(x[b]), tokens[b].tolist(), f64(u[b]), f64(q[b]) if drafted else None,
                                                    None, float(_temps(1, t)[0]))
        if margin < 2.0 ** -16:
            continue
        clear += 1
        assert r.tokens[b].tolist() == ids + [-1] * (2 - len(ids)), b
        assert np.abs(f64(r.logprobs[b])[: len(ids)] - logps).max() <= 2.0 ** -18
    assert clear >= 0.9 * B


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("t", [1e30, 3e38])
def test_bad_rows_stay_bad_at_high_temperatures(cuda_device, bad, t):
    x = torch.full((3, 5001), NEG, device=DEV)
    x[1, 4000] = bad
    status = w.new_status(DEV)
    r = w.token_logprobs(x, torch.zeros(3, 1, dtype=torch.int32, device=DEV), top_k=1, temperature=_temps(3, t), status=status)
    assert int(status.item()) == L.DEV_LOGITS
    assert r.lse[1].isnan() and r.top_ids[:, 0].tolist() == [-1] * 3 and r.lse[::2].tolist() == [NEG] * 2


LOW_BAD = [1e-45, 1e-39, 2.9e-39, 3e-39, 4e-39, 4.2e-39]  # 1 / T or log2(e) / T pass fp32


@pytest.mark.parametrize("t", LOW_BAD)
@pytest.mark.parametrize("vocab", [3, 5001, 131072])
def test_temperatures_below_the_lowest_are_bad(cuda_device, t, vocab):
    """Whatever the row holds: logits, or masked tokens alone."""
    x = torch.randn(3, vocab, device=DEV)
    x[1], x[2] = NEG, 0.0
    status = w.new_status(DEV)
    r = w.token_logprobs(x, torch.zeros(3, 1, dtype=torch.int32, device=DEV), top_k=2, temperature=_temps(3, t), status=status)
    assert int(status.item()) == L.DEV_LOGITS
    assert r.lse.isnan().all() and r.entropy.isnan().all() and r.logprobs.isnan().all() and r.top_logprobs.isnan().all()
    assert (r.top_ids == -1).all()
    status.zero_()
    none = torch.zeros(3, 0, dtype=torch.int32, device=DEV)
    a = w.accept_draft(x[:, None], none, torch.full((3, 1), 0.5, device=DEV), temperature=_temps(3, t), status=status)
    assert int(status.item()) == L.DEV_LOGITS and (a.count == 0).all() and (a.tokens == -1).all()


@pytest.mark.parametrize("t", [4.25e-39, 5e-39, 1.1e-38, 1.2e-38, 1e-30])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("vocab", [3, 5001, 131072])
def test_lowest_temperatures(cuda_device, t, dtype, vocab):
    """The largest logit has all the weight.  A log probability is (x - max) / T with three roundings: 1 / T is a normal
    number although T is not."""
    x = torch.full((3, vocab), -0.125, device=DEV)
    x[0, vocab - 1] = x[1, 1] = 0.0
    x[2] = NEG
    x[2, 2] = 0.5
    x = x.to(DT[dtype])
    best = [vocab - 1, 1, 2]
    ids = torch.tensor([[b, 0] for b in best], dtype=torch.int32, device=DEV)
    status = w.new_status(DEV)
    r = w.token_logprobs(x, ids, top_k=1, temperature=_temps(3, t), status=status)
    assert r.top_ids[:, 0].tolist() == best and (r.logprobs[:, 0] == 0).all() and (r.entropy == 0).all()
    want = -0.125 / float(_temps(1, t)[0])
    assert np.abs(f64(r.logprobs[:2, 1]) - want).max() <= 3 * 2.0 ** -24 * abs(want) and r.logprobs[2, 1] == NEG
    drafts = torch.tensor([[best[0]], [0], [best[2]]], dtype=torch.int32, device=DEV)
    a = w.accept_draft(x[:, None].expand(3, 2, vocab), drafts, torch.full((3, 2), 0.75, device=DEV),
                       temperature=_temps(3, t), status=status)
    assert int(status.item()) == 0
    assert a.tokens.tolist() == [[best[0]] * 2, [1, -1], [2, 2]] and (a.logprobs == 0).all()
