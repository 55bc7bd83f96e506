"""token_logprobs and accept_draft against the fp64 oracle.

Tolerances.  y = (x - max) / T is rounded three times (1 / T, the difference,
the product): 3 * 2^-24 |y|.  A row's sum S = sum exp(y) of N columns: each term
is off by 2^-22 (the hardware's 2^x) and by its argument's error; a thread adds at
most N / 256 + 40 terms or partial sums in a row, each addition off by 2^-24.
So S is off by e_S = 2^-22 + (N / 256 + 40) 2^-24 + 4 * 2^-24 E|y|, E|y| the mean of
|y| under the row's distribution; ln S by e_S and one ulp of logf; a log
probability by that and 3 * 2^-24 |y|, the log-sum-exp by that and one rounding
each of max / T and the sum; and the entropy, whose two sums have terms e and e y,
by (1 + E|y|) e_S, 4 * 2^-24 E y^2 (terms e y moved by their argument) and the
roundings of its value.
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
U = 2.0 ** -24
NEG = float("-inf")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _tolerances(row, t):
    y = (row - row.max()) / t
    p = np.exp(y)
    p /= p.sum()
    there = p > 0
    mean, square = -(p[there] * y[there]).sum(), (p[there] * y[there] ** 2).sum()
    e_s = 2.0 ** -22 + (len(row) / 256 + 40) * U + 4 * U * mean
    lse = abs(row.max() / t)
    ln = abs(np.log(np.exp(y[y > -np.inf]).sum()))
    return e_s + 2 * U * ln, e_s + 2 * U * ln + 4 * U * (lse + ln), (1 + mean) * e_s + 4 * U * square + 6 * U * (ln + mean), y


def _check_rows(x, tokens, top_k, temperature, r):
    lp, ent, lse = f64(r.logprobs), f64(r.entropy), f64(r.lse)
    x64, toks = f64(x), tokens.cpu().numpy()
    temps = np.ones(len(x64)) if temperature is None else f64(temperature)
    for i, row in enumerate(x64):
        ref, ref_lse, ref_ent = oracle.row_logprobs(row, temps[i])
        if ref_lse == -np.inf:
            assert lse[i] == -np.inf and ent[i] == 0 and (lp[i] == -np.inf).all()
        else:
            tol, tol_lse, tol_ent, y = _tolerances(row, temps[i])
            assert abs(lse[i] - ref_lse) <= tol_lse, (i, lse[i], ref_lse, tol_lse)
            assert abs(ent[i] - ref_ent) <= tol_ent, (i, ent[i], ref_ent, tol_ent)

            def close(got, ids):
                for a, j in zip(got, ids):
                    want = ref[j] if 0 <= j < len(row) else -np.inf
                    if want <= -2.0 ** 128:  # beyond fp32, which rounds it to -inf
                        assert a == -np.inf
                    else:
                        assert abs(a - want) <= tol + 3 * U * abs(y[j]) + U * abs(want), (i, j, a, want)
            close(lp[i], toks[i])
        if top_k:
            ids = oracle.top_tokens(row, top_k)
            assert r.top_ids[i].tolist() == ids
            close(f64(r.top_logprobs[i]), ids) if ref_lse > -np.inf else None


def _case(seed, rows, vocab, dtype, given=2, top=5, temperature=False, slack=0, masked=0.0, coarse=False):
    g = _gen(seed)
    x = torch.randn(rows, vocab + slack, generator=g, device=DEV) * 3
    if coarse:  # many equal logits
        x = x.round()
    x = x.to(DT[dtype])
    if masked:
        x.masked_fill_(torch.rand(x.shape, generator=g, device=DEV) < masked, NEG)
    x[:, vocab:] = float("nan")
    tokens = torch.randint(0, vocab, (rows, given), generator=g, device=DEV).int()
    t = torch.rand(rows, generator=g, device=DEV) * 2 + 0.1 if temperature else None
    status = w.new_status(DEV)
    r = w.token_logprobs(x[:, :vocab], tokens, top_k=top, temperature=t, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    _check_rows(x[:, :vocab], tokens, top, t, r)


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 63, 511, 513, 4096, 5003, 50257])
@pytest.mark.parametrize("dtype", list(DT))
def test_logprob_vocabularies(cuda_device, vocab, dtype):
    _case(vocab, 3, vocab, dtype, top=min(vocab, 20))


@pytest.mark.parametrize("rows,vocab", [(1, 131072), (4, 129281), (40, 30001), (200, 9973), (700, 1500)])
@pytest.mark.parametrize("kw", [dict(top=64, temperature=True), dict(top=0, given=0), dict(top=1, given=9, slack=3, masked=0.9),
                                dict(top=20, slack=1, dtype="fp32", coarse=True)])
def test_logprob_rows(cuda_device, rows, vocab, kw):
    _case(rows, rows, vocab, **{"dtype": "bf16", **kw})


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("top", [1, 33, 64])
def test_logprob_ties_and_runs(cuda_device, dtype, top):
    """Equal logits everywhere, the largest in one run of columns, sorted both ways."""
    V = 20011
    rows = torch.zeros(7, V, device=DEV)
    rows[1, 5000:5200] = 4.0
    rows[2] = torch.linspace(-5, 5, V, device=DEV)
    rows[3] = torch.linspace(5, -5, V, device=DEV)
    rows[4, ::512] = 3.0
    rows[5] = NEG
    rows[5, [3, 17, V - 1]] = torch.tensor([1.0, 2.0, 1.0], device=DEV)
    rows[6, :8] = -1.0
    x = rows.to(DT[dtype])
    tokens = torch.tensor([[0, V - 1]] * 7, dtype=torch.int32, device=DEV)
    status = w.new_status(DEV)
    _check_rows(x, tokens, top, None, w.token_logprobs(x, tokens, top_k=top, status=status))
    assert int(status.item()) == 0


def test_logprob_masked_and_extreme_rows(cuda_device):
    V = 3000
    low = torch.finfo(torch.float32).min
    x = torch.zeros(6, V, device=DEV)
    x[0] = NEG
    x[1] = low  # masked with the type's lowest value, all of them
    x[2], x[2, 7] = low, 0.5
    x[3], x[3, 9] = NEG, 1e30
    x[4], x[4, 11] = 1e30, NEG
    x[5] = torch.linspace(-300, 300, V, device=DEV)
    tokens = torch.tensor([[0, 7, 9, 11, -1]] * 6, dtype=torch.int32, device=DEV)
    status = w.new_status(DEV)
    r = w.token_logprobs(x, tokens, top_k=3, status=status)
    assert int(status.item()) == 0
    lp = r.logprobs
    assert (lp[:, 4] == NEG).all()
    assert (lp[0] == NEG).all() and r.lse[0] == NEG and r.entropy[0] == 0 and r.top_ids[0].tolist() == [-1] * 3
    assert (r.top_logprobs[0] == NEG).all()
    want = -np.log(V)
    assert abs(float(lp[1, 0]) - want) < 1e-5 and abs(float(r.entropy[1]) + want) < 1e-5
    assert r.top_ids[1].tolist() == [0, 1, 2]
    assert lp[2, 1] == 0 and lp[2, 0] == low - 0.5 and r.entropy[2] == 0 and r.top_ids[2].tolist() == [7, 0, 1]
    assert lp[3, 2] == 0 and lp[3, 0] == NEG and r.top_ids[3].tolist() == [9, -1, -1]
    assert abs(float(lp[4, 0]) + np.log(V - 1)) < 1e-5 and lp[4, 3] == NEG
    _check_rows(x[5:], tokens[5:], 3, None, w.token_logprobs(x[5:], tokens[5:], top_k=3))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [2, 700])
def test_logprob_top_tokens_among_very_many_equal_ones(cuda_device, dtype, rows):
    """Fewer tokens than top_k above a plain of equal logits; a few in one thread's columns; a plain above all."""
    V, top = 40003, 64
    x = torch.full((rows, V), -1e4, device=DEV)
    x[0, torch.randperm(V, generator=_gen(40), device=DEV)[:20]] = torch.randn(20, generator=_gen(41), device=DEV)
    x[1, 8192 * torch.arange(4, device=DEV) + 3] = 2.0
    if rows > 2:
        x[2:] = torch.randn(rows - 2, V, generator=_gen(42), device=DEV)
        x[2, 10000:20000] = 9.0
        x[3, 5::2048] = 9.0
        x[4] = NEG
        x[4, 30000:30040] = 1.0
        x[5] = NEG
        x[5, 17:30000] = torch.finfo(DT[dtype]).min
        x[6, 100:3000] = torch.linspace(20, 40, 2900, device=DEV)
    x = x.to(DT[dtype])
    tokens = torch.zeros(rows, 1, dtype=torch.int32, device=DEV)
    r = w.token_logprobs(x, tokens, top_k=top)
    for i in range(min(rows, 9)):
        assert r.top_ids[i].tolist() == oracle.top_tokens(f64(x[i]), top), i


def test_logprob_top_tokens_all_in_few_columns_of_a_stride(cuda_device):
    """Thousands of the largest logits where one thread in 64 looks: every column of 8 in 2048."""
    R, V = 1000, 131072
    x = torch.randn(R, V, generator=_gen(43), device=DEV).bfloat16()
    big = (torch.arange(V, device=DEV) % 2048) < 32
    x[5, big] = (torch.rand(int(big.sum()), generator=_gen(44), device=DEV) * 50 + 10).bfloat16()
    r = w.token_logprobs(x, torch.zeros(R, 1, dtype=torch.int32, device=DEV), top_k=64)
    for i in (4, 5, 6):
        assert r.top_ids[i].tolist() == oracle.top_tokens(f64(x[i]), 64)


@pytest.mark.parametrize("t", [1e-30, 1e-6, 0.01, 100.0, 1e6, 1e30])
@pytest.mark.parametrize("masked", [False, True])
def test_logprob_extreme_temperatures(cuda_device, t, masked):
    x = torch.randn(4, 5001, generator=_gen(20), device=DEV)
    if masked:
        x[:, ::3] = NEG
        x[3, 1:] = NEG
        x[3, 0] = 1.0
    tokens = torch.tensor([[0, 1, 5000]] * 4, dtype=torch.int32, device=DEV)
    temps = torch.full((4,), t, device=DEV)
    status = w.new_status(DEV)
    r = w.token_logprobs(x, tokens, top_k=4, temperature=temps, status=status)
    assert int(status.item()) == 0
    if t == 1e-30:  # all but the largest underflow; the others' log probabilities pass fp32 or not
        assert (r.entropy == 0).all() and (r.top_logprobs[:, 0] == 0).all()
        assert r.top_ids.tolist() == [oracle.top_tokens(row, 4) for row in f64(x)]
        return
    _check_rows(x, tokens, 4, temps, r)


@pytest.mark.parametrize("dtype,shift", [("fp32", 3e5), ("fp32", -3e5), ("fp32", 1e7), ("fp32", 1e20), ("fp32", -1e35),
                                         ("fp16", 6e4), ("fp16", -6e4), ("bf16", 3e5), ("bf16", -1e38), ("bf16", 2e38)])
def test_logprob_large_logits(cuda_device, dtype, shift):
    """Far from 0: differences keep their digits."""
    g = _gen(21)
    step = abs(shift) * torch.finfo(DT[dtype]).eps
    x = (shift + torch.randint(-6, 7, (3, 4007), generator=g, device=DEV) * step).to(DT[dtype])
    x[1, 7:900] = NEG
    t = torch.full((3,), max(1.0, step), device=DEV)
    tokens = torch.randint(0, 4007, (3, 3), generator=g, device=DEV).int()
    status = w.new_status(DEV)
    r = w.token_logprobs(x, tokens, top_k=3, temperature=t, status=status)
    assert int(status.item()) == 0
    _check_rows(x, tokens, 3, t, r)


def test_logprob_offsets_beyond_32_bits(cuda_device):
    R, V = 17000, 131072  # 2.2e9 logits
    x = torch.zeros(R, V, dtype=torch.bfloat16, device=DEV)
    last = torch.randn(3, V, generator=_gen(22), device=DEV).bfloat16()
    x[-3:] = last
    tokens = torch.full((R, 1), 77, dtype=torch.int32, device=DEV)
    r = w.token_logprobs(x, tokens, top_k=2)
    assert (r.logprobs[:-3] + np.log(V)).abs().max() < 1e-5 and (r.top_ids[:-3] == torch.tensor([0, 1], device=DEV)).all()
    _check_rows(last, tokens[-3:], 2, None, w.TokenLogprobs(r.logprobs[-3:], r.entropy[-3:], r.lse[-3:],
                                                            r.top_logprobs[-3:], r.top_ids[-3:]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("col", [0, 1, 4097, 9000])
def test_logprob_rows_without_a_distribution(cuda_device, bad, col):
    x = torch.randn(3, 9001, generator=_gen(3), device=DEV)
    x[1, col] = bad
    tokens = torch.zeros(3, 1, dtype=torch.int32, device=DEV)
    status = w.new_status(DEV)
    r = w.token_logprobs(x, tokens, top_k=2, status=status)
    assert int(status.item()) == L.DEV_LOGITS
    for t in (r.logprobs[1], r.entropy[1:2], r.lse[1:2], r.top_logprobs[1]):
        assert t.isnan().all()
    assert r.top_ids[1].tolist() == [-1, -1]
    ok = w.token_logprobs(x[::2].contiguous(), tokens[::2].contiguous(), top_k=2)
    assert torch.equal(r.logprobs[::2], ok.logprobs) and torch.equal(r.top_ids[::2], ok.top_ids)


def test_logprob_bad_temperatures_and_tokens(cuda_device):
    x = torch.randn(6, 100, generator=_gen(4), device=DEV)
    t = torch.tensor([1.0, 0.0, -1.0, float("nan"), float("inf"), 2.0], device=DEV)
    tokens = torch.tensor([[5]] * 6, dtype=torch.int32, device=DEV)
    status = w.new_status(DEV)
    r = w.token_logprobs(x, tokens, top_k=1, temperature=t, status=status)
    assert int(status.item()) == L.DEV_LOGITS
    assert r.lse.isnan().tolist() == [False, True, True, True, True, False]
    status.zero_()
    ids = torch.tensor([[-1], [100], [-2], [0], [99], [1 << 30]], dtype=torch.int32, device=DEV)
    r = w.token_logprobs(x, ids, status=status)
    assert int(status.item()) == L.DEV_TOKEN_OOB
    assert (r.logprobs[:, 0] == NEG).tolist() == [True, True, True, False, False, True]
    assert r.top_ids is None and r.top_logprobs is None


def test_logprob_same_bits_alone_and_in_a_batch(cuda_device):
    x = torch.randn(9, 40000, generator=_gen(5), device=DEV).bfloat16()
    tokens = torch.randint(0, 40000, (9, 3), generator=_gen(6), device=DEV).int()
    a, b = (w.token_logprobs(x, tokens, top_k=9) for _ in range(2))
    for n in ("logprobs", "entropy", "lse", "top_logprobs", "top_ids"):
        assert torch.equal(getattr(a, n), getattr(b, n))


def test_logprob_empty_and_refusals(cuda_device):
    x = torch.randn(4, 64, device=DEV)
    i = torch.zeros(4, 1, dtype=torch.int32, device=DEV)
    r = w.token_logprobs(x[:0], i[:0], top_k=2)
    assert r.logprobs.shape == (0, 1) and r.top_ids.shape == (0, 2)
    for err, args, kw in [
        (TypeError, (x.double(), i), {}),
        (TypeError, (x, i.long()), {}),
        (ValueError, (x, i[:2]), {}),
        (ValueError, (x.t(), i), {}),
        (ValueError, (x, i), dict(temperature=torch.ones(3, device=DEV))),
        (ValueError, (x, i), dict(top_k=-1)),
        (w.WmtpError, (x, i), dict(top_k=65)),
        (w.WmtpError, (x[:1].expand(4, 64), i), {}),
        (ValueError, (x, i.cpu()), {}),
    ]:
        with pytest.raises(err):
            w.token_logprobs(*args, **kw)


# ---------------------------------------------------------------- acceptance
def _accept_case(seed, batch, gamma, vocab, dtype, drafted, greedy=0, ragged=False, slack=0, masked=0.0, spread=3.0):
    g = _gen(seed)
    dt = DT[dtype]
    target = (torch.randn(batch, gamma + 1, vocab + slack, generator=g, device=DEV) * spread).to(dt)[..., :vocab]
    draft = (target[:, :gamma].float() + torch.randn(batch, gamma, vocab, generator=g, device=DEV) * 0.7).to(dt)
    if masked:
        gone = torch.rand(target.shape, generator=g, device=DEV) < masked
        gone[..., 0] = False
        target.masked_fill_(gone, NEG)
    noise = -torch.log(-torch.log(torch.rand(draft.shape, generator=g, device=DEV).clamp(1e-12)))
    tokens = (draft.float() + noise).argmax(-1).int() if drafted else draft.argmax(-1).int()
    t = torch.rand(batch, generator=g, device=DEV) + 0.5
    if greedy:
        t[::greedy] = 0
    num = torch.randint(0, gamma + 1, (batch,), generator=g, device=DEV).int() if ragged else None
    u = torch.rand(batch, gamma + 1, generator=g, device=DEV)
    status = w.new_status(DEV)
    r = w.accept_draft(target, tokens, u, draft_logits=draft if drafted else None, num_draft=num, temperature=t,
                       status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    clear = 0
    for b in range(batch):
        ids, logps, margin = oracle.accept_sequence(
            f64(target[b]), tokens[b].tolist(), f64(u[b]), f64(draft[b]) if drafted else None,
            None if num is None else int(num[b]), float(t[b]))
        if margin < 1e-5:  # decided by less than the roundings of the distributions
            continue
        clear += 1
        n = len(ids)
        assert int(r.count[b]) == n and r.tokens[b].tolist() == ids + [-1] * (gamma + 1 - n), (b, margin)
        lp = f64(r.logprobs[b])
        assert (lp[n:] == 0).all()
        for i in range(n):
            row = f64(target[b, i])
            tol, _, _, y = _tolerances(row, float(t[b]) or 1.0)
            assert abs(lp[i] - logps[i]) <= tol + 3 * U * abs(y[ids[i]]) + U * abs(logps[i])
    assert clear >= 0.9 * batch


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("vocab", [1, 2, 9, 513, 5003, 40001])
def test_accept_vocabularies(cuda_device, vocab, dtype, drafted):
    _accept_case(vocab, 6, 3, vocab, dtype, drafted)


@pytest.mark.parametrize("batch,gamma,vocab", [(1, 0, 1000), (1, 1, 131072), (3, 8, 20000), (40, 5, 3001), (130, 2, 700),
                                               (2, 31, 600)])
@pytest.mark.parametrize("kw", [dict(drafted=True, greedy=3, ragged=True, slack=5), dict(drafted=False, greedy=2, masked=0.8),
                                dict(drafted=True, masked=0.5, spread=0.5)])
def test_accept_batches(cuda_device, batch, gamma, vocab, kw):
    _accept_case(batch, batch, gamma, vocab, "bf16", **kw)


def test_accepted_tokens_follow_the_target(cuda_device):
    """The first emitted token is distributed as the target's first row, and the token behind one accepted draft as
    its second, whatever the drafts: counts within five standard deviations."""
    N, V = 40000, 7
    g = _gen(8)
    target = (torch.randn(1, 2, V, generator=g, device=DEV) * 1.5).expand(N, 2, V)
    draft = (torch.randn(1, 1, V, generator=g, device=DEV) * 1.5).expand(N, 1, V)
    q = torch.softmax(draft[0, 0], 0)
    tokens = torch.multinomial(q, N, replacement=True, generator=g).int()[:, None]
    r = w.accept_draft(target, tokens, torch.rand(N, 2, generator=g, device=DEV), draft_logits=draft)
    p = f64(torch.softmax(target[0].double(), -1))
    assert 0.1 * N < int((r.count == 2).sum()) < 0.95 * N
    for i, sel in ((0, r.count >= 1), (1, r.count == 2)):
        n = int(sel.sum())
        seen = np.bincount(r.tokens[sel, i].cpu().numpy(), minlength=V)
        assert (np.abs(seen - n * p[i]) < 5 * np.sqrt(n * p[i] * (1 - p[i])) + 1).all()


def test_accept_extreme_draws(cuda_device):
    """u of 0 and just below 1 take the first and last token that has any weight."""
    V = 5000
    x = torch.full((2, 1, V), NEG, device=DEV)
    x[:, 0, 100:4000] = torch.randn(3900, generator=_gen(9), device=DEV)
    none = torch.zeros(2, 0, dtype=torch.int32, device=DEV)
    u = torch.tensor([[0.0], [1.0 - 2.0 ** -24]], device=DEV)
    r = w.accept_draft(x, none, u)
    first, last = r.tokens[:, 0].tolist()
    assert first == 100 and 3990 <= last < 4000 and r.count.tolist() == [1, 1]
    ids, _, _ = oracle.accept_sequence(f64(x[1]), [], f64(u[1]))
    assert last == ids[0]


def test_accept_draft_that_takes_all_weight(cuda_device):
    """A rejected draft whose distribution covers the target's everywhere it can: only the rest is drawn."""
    V = 300
    x = torch.full((2, 2, V), NEG, device=DEV)
    x[0, :, 7] = 0.0  # one token: drafted, so accepted whatever u
    x[1, :, [7, 200]] = 0.0
    tokens = torch.tensor([[7], [9]], dtype=torch.int32, device=DEV)
    u = torch.full((2, 2), 0.75, device=DEV)
    r = w.accept_draft(x, tokens, u)
    assert r.tokens.tolist() == [[7, 7], [200, -1]]
    q = x[:, :1].clone()
    q[1, 0] = NEG
    q[1, 0, 9] = 0.0
    r = w.accept_draft(x, tokens, u, draft_logits=q)
    assert r.tokens.tolist() == [[7, 7], [200, -1]]


def test_accept_bad_rows_lengths_and_ids(cuda_device):
    B, G, V = 9, 2, 600
    x = torch.zeros(B, G + 1, V, device=DEV)
    x[..., 5] = 20.0
    tokens = torch.full((B, G), 5, dtype=torch.int32, device=DEV)
    u = torch.full((B, G + 1), 0.5, device=DEV)
    t = torch.ones(B, device=DEV)
    num = torch.full((B,), G, dtype=torch.int32, device=DEV)
    x[0, 1, 3] = float("nan")
    x[1, 2, 4] = float("inf")
    x[2, 0] = NEG
    t[3], t[4] = -1.0, float("nan")
    num[5], num[6] = -1, 3
    tokens[7, 1], tokens[8, 0] = V, -1
    status = w.new_status(DEV)
    r = w.accept_draft(x, tokens, u, num_draft=num, temperature=t, status=status)
    assert int(status.item()) == L.DEV_LOGITS | L.DEV_LEN_OOB | L.DEV_TOKEN_OOB
    assert r.count.tolist() == [1, 2, 0, 0, 0, 0, 0, 2, 1]
    assert r.tokens[:3].tolist() == [[5, -1, -1], [5, 5, -1], [-1] * 3]
    assert r.tokens[7].tolist() == [5, 5, -1] and r.tokens[8].tolist() == [5, -1, -1]
    # rows that are not needed may hold anything
    x[:] = float("nan")
    x[:, 0] = 0.0
    x[:, 0, 5] = 20.0
    status.zero_()
    r = w.accept_draft(x, tokens, u, num_draft=torch.zeros_like(num), status=status)
    assert int(status.item()) == 0 and r.count.tolist() == [1] * B and (r.tokens[:, 0] == 5).all()


def test_accept_same_distributions_accept_everything(cuda_device):
    x = torch.randn(50, 4, 3001, generator=_gen(30), device=DEV).half()
    tokens = torch.randint(0, 3001, (50, 3), generator=_gen(31), device=DEV).int()
    u = torch.rand(50, 4, generator=_gen(32), device=DEV)
    r = w.accept_draft(x, tokens, u, draft_logits=x[:, :3])
    assert (r.count == 4).all() and torch.equal(r.tokens[:, :3], tokens)


@pytest.mark.parametrize("dtype,mask", [(d, m) for d in DT for m in (-1e4, -1e9, -1e10, -1e25, "lowest")
                                        if d != "fp16" or m in (-1e4, "lowest")])
@pytest.mark.parametrize("t", [0.05, 4.0])
def test_accept_masks_that_are_finite(cuda_device, dtype, mask, t):
    """Tokens masked with a large negative logit, whole runs of them, are never drawn."""
    B, V = 40, 9001
    x = torch.randn(B, 3, V, generator=_gen(33), device=DEV).to(DT[dtype])
    allowed = torch.zeros(V, dtype=torch.bool, device=DEV)
    allowed[5::7] = True
    allowed[1000:6000] = False
    x[:, :, ~allowed] = torch.finfo(DT[dtype]).min if mask == "lowest" else mask
    q = torch.randn(B, 2, V, generator=_gen(34), device=DEV).to(DT[dtype])
    tokens = torch.randint(0, V, (B, 2), generator=_gen(35), device=DEV).int()
    u = torch.rand(B, 3, generator=_gen(36), device=DEV)
    status = w.new_status(DEV)
    r = w.accept_draft(x, tokens, u, draft_logits=q, temperature=torch.full((B,), t, device=DEV), status=status)
    assert int(status.item()) == 0
    out = r.tokens[r.tokens >= 0].long()
    assert allowed[out].all() and (r.count >= 1).all()
    temps = torch.full((B,), t, device=DEV)
    ids = tokens[:, :1].contiguous()
    _check_rows(x[:3, 0].contiguous(), ids[:3], 5, temps[:3], w.token_logprobs(x[:3, 0].contiguous(), ids[:3], top_k=5,
                                                                               temperature=temps[:3]))


def test_accept_broadcast_and_refusals(cuda_device):
    x = torch.randn(2, 3, 50, generator=_gen(10), device=DEV)
    tokens = torch.tensor([[1, 2], [3, 4]], dtype=torch.int32, device=DEV)
    u = torch.rand(2, 3, generator=_gen(11), device=DEV)
    one = x[:1].expand(2, 3, 50)
    a, b = w.accept_draft(one, tokens, u), w.accept_draft(one.contiguous(), tokens, u)
    assert torch.equal(a.tokens, b.tokens) and torch.equal(a.logprobs, b.logprobs)
    assert w.accept_draft(x[:0], tokens[:0], u[:0]).tokens.shape == (0, 3)
    for err, args, kw in [
        (TypeError, (x.double(), tokens, u), {}),
        (ValueError, (x[0], tokens, u), {}),
        (ValueError, (x, tokens[:, :1], u), {}),
        (ValueError, (x, tokens, u[:, :2]), {}),
        (TypeError, (x, tokens.long(), u), {}),
        (TypeError, (x, tokens, u), dict(draft_logits=x[:, :2].bfloat16())),
        (ValueError, (x, tokens, u), dict(draft_logits=x)),
        (ValueError, (x.transpose(1, 2), tokens, u), {}),
        (ValueError, (x, tokens, u), dict(temperature=torch.ones(3, device=DEV))),
        (w.WmtpError, (torch.zeros(1, 33, 8, device=DEV), torch.zeros(1, 32, dtype=torch.int32, device=DEV),
                       torch.zeros(1, 33, device=DEV)), {}),
    ]:
        with pytest.raises(err):
            w.accept_draft(*args, **kw)
