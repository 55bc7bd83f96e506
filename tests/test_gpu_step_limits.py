"""token_logprobs and accept_draft at the ends of the temperatures' range.

At a temperature T of 1e28 and above every finite logit of ordinary size has the same weight; a masked one has
none at any temperature.  Where one token is left its log probability is exactly 0, as ln 1 and 0 / T are.
"""

import pytest
import torch

import speculative_decode_draft_b200 as w
from speculative_decode_draft_b200 import _lib as L

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


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("t", [1e30, 3e38])
def test_bad_rows_stay_bad_at_high_temperatures(cuda_device, bad, t):
    x = torch.full((3, 5001), NEG, device=DEV)
    x[1, 4000] = bad
    status = w.new_status(DEV)
    r = w.token_logprobs(x, torch.zeros(3, 1, dtype=torch.int32, device=DEV), top_k=1, temperature=_temps(3, t), status=status)
    assert int(status.item()) == L.DEV_LOGITS
    assert r.lse[1].isnan() and r.top_ids[:, 0].tolist() == [-1] * 3 and r.lse[::2].tolist() == [NEG] * 2
