"""Pins of oracle/step.py: properties that follow from the definitions."""

import numpy as np
import pytest

import oracle
import speculative_decode_draft_b200 as w


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_scores_depend_on_the_distance(interleaved):
    rng = np.random.default_rng(1)
    freq = w.rope_frequencies(8, 100.0)
    q, k = rng.standard_normal((2, 1, 1, 12))

    def score(t, s):
        a = oracle.rotate_heads(q, [t], freq, interleaved=interleaved)
        b = oracle.rotate_heads(k, [s], freq, interleaved=interleaved)
        assert np.allclose(np.linalg.norm(a), np.linalg.norm(q))
        assert np.array_equal(a[..., 8:], q[..., 8:])  # behind the rotated part
        return (a * b).sum()
    assert np.isclose(score(7, 3), score(1000007, 1000003), atol=1e-9)
    assert not np.isclose(score(7, 3), score(7, 4), atol=1e-3)
    assert np.allclose(oracle.rotate_heads(q, [0], freq, interleaved=interleaved), q)


def test_rotation_of_one_pair_by_a_quarter_turn():
    x = np.array([[[3.0, 5.0, 2.0, 7.0]]])
    quarter = [np.pi / 2, np.pi]
    assert np.allclose(oracle.rotate_heads(x, [1], quarter), [[[-2.0, -5.0, 3.0, -7.0]]])
    assert np.allclose(oracle.rotate_heads(x, [1], quarter, interleaved=True, factor=2.0), [[[-10.0, 6.0, -4.0, -14.0]]])


def test_head_norm_has_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((3, 2, 16)) * 5
    y = oracle.rotate_heads(x, [0, 1, 2], [], weight=np.zeros(16), offset=1.0, eps=0.0)
    assert np.allclose((y ** 2).mean(-1), 1.0)


def test_frequencies_by_scaling():
    plain = w.rope_frequencies(64, 1e4)
    assert plain[0] == 1.0 and np.isclose(plain[-1], 1e4 ** (-62 / 64))
    assert np.allclose(w.rope_frequencies(64, 1e4, scaling="linear", stretch=8.0), np.array(plain) / 8)
    for scaling in ("yarn", "bands"):
        f = np.array(w.rope_frequencies(64, 1e4, scaling=scaling, stretch=4.0, original=4096))
        r = f / plain
        assert r[0] == 1.0 and np.isclose(r[-1], 0.25) and (np.diff(r) <= 1e-15).all()
        assert ((r > 0.25) & (r < 1.0)).any()
    for bad in (dict(scaling="yarn"), dict(scaling="bands", original=5, fast=1.0, slow=2.0), dict(scaling="what"),
                dict(scaling="linear", stretch=0.0)):
        with pytest.raises(ValueError):
            w.rope_frequencies(64, **bad)
    with pytest.raises(ValueError):
        w.rope_frequencies(7)


def test_page_model_keeps_every_page_once():
    rng = np.random.default_rng(3)
    P, pages, B, width = 16, 40, 5, 12
    m = oracle.PageModel(P, pages, np.full((B, width), -1), np.zeros(B, int), range(pages))
    for _ in range(200):
        before = list(m.kv_len)
        new = rng.integers(-1, width * P + 2, B)
        cu, pos, slots, wrong = m.resize(new, 100)
        held = [p for b in range(B) for p in m.table[b] if p >= 0]
        assert sorted(held + m.free) == list(range(pages))
        for b in range(B):
            n = -(-m.kv_len[b] // P)
            assert all(p >= 0 for p in m.table[b][:n]) and all(p < 0 for p in m.table[b][n:])
            assert cu[b + 1] - cu[b] == max(m.kv_len[b] - before[b], 0)
        assert len(set(slots[: cu[-1]])) == cu[-1] and ("len" in wrong) == any(x < 0 or x > width * P for x in new)


def test_growth_taken_back_leaves_the_stack():
    m = oracle.PageModel(16, 30, np.full((2, 8), -1), [0, 0], range(30))
    m.resize([20, 50])
    table, free = [list(r) for r in m.table], list(m.free)
    m.resize([100, 128])
    m.resize([20, 50])
    assert m.table == table and m.free == free


def test_logprobs_sum_to_one_and_masked_rows():
    lp, lse, h = oracle.row_logprobs([1.0, 2.0, -np.inf], 0.5)
    assert np.isclose(np.exp(lp).sum(), 1.0) and lp[2] == -np.inf and np.isclose(lse, np.log(np.exp(2) + np.exp(4)))
    assert np.isclose(h, -(np.exp(lp[:2]) * lp[:2]).sum())
    lp, lse, h = oracle.row_logprobs([-np.inf, -np.inf])
    assert lse == -np.inf and h == 0.0
    assert oracle.top_tokens([1.0, 3.0, 3.0, -np.inf], 4) == [1, 2, 0, -1]


@pytest.mark.parametrize("with_draft", [False, True])
def test_emitted_tokens_follow_the_target(with_draft):
    rng = np.random.default_rng(4)
    V, N = 5, 20000
    target, draft = rng.standard_normal((2, V)) * 1.5, rng.standard_normal((1, V)) * 1.5
    p = np.exp(oracle.row_logprobs(target[0])[0])
    q = np.exp(oracle.row_logprobs(draft[0])[0])
    seen = np.zeros(V)
    for _ in range(N):
        d = rng.choice(V, p=q) if with_draft else 2
        seen[oracle.accept_sequence(target, [d], rng.random(2), draft if with_draft else None)[0][0]] += 1
    # each count is binomial: five standard deviations
    assert (np.abs(seen - N * p) < 5 * np.sqrt(N * p * (1 - p))).all()
