"""qk_norm_rope against the fp64 oracle.

Tolerance: the result is rounded to bf16 once (half a step, 2^-8 of the value,
torch.finfo(bf16).eps / 2).  Before it everything is fp32: the sum of D squares
over lanes (at most 8 + 5 additions in a row, 13 * 2^-24), rsqrt (2 ulp), three
products, and cos and sin with an angle that is off by 2^-25 half turns
(pi 2^-25) plus 2 ulp: below 32 * 2^-24 = 2^-19 of factor * (|a| + |b|) of the
pair.
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
BF16, F32 = torch.bfloat16, torch.float32


def _pair_sum(y, n, interleaved, factor):
    """factor (|a| + |b|) of each element's pair, |y| where it is not rotated."""
    s = np.abs(y).copy()
    first = np.arange(n) * 2 if interleaved else np.arange(n)
    second = first + 1 if interleaved else first + n
    s[..., first] = s[..., second] = np.abs(factor) * (np.abs(y[..., first]) + np.abs(y[..., second]))
    return s


def _check(got, x, positions, freq, weight, offset, eps, interleaved, factor, what):
    w64 = None if weight is None else f64(weight)
    ref = oracle.rotate_heads(f64(x), positions, freq, interleaved=interleaved, factor=factor, weight=w64, offset=offset,
                              eps=eps)
    normed = oracle.rotate_heads(f64(x), positions, [], weight=w64, offset=offset, eps=eps)
    tol = 2.0 ** -8 * np.abs(ref) + 1.01 * 2.0 ** -19 * _pair_sum(normed, len(freq), interleaved, factor) + 1e-38
    bad = np.abs(f64(got) - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}"


def _run(seed, tokens, heads, kv_heads, dim, rotary, *, page=16, interleaved=False, factor=1.0, norm=True, offset=0.0,
         eps=1e-6, dtype=BF16, wdtype=F32, packed=False, far=1 << 20, pad=0, base=1e4):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    if packed:
        qkv = torch.randn(tokens, (heads + 2 * kv_heads) * dim, generator=g, device=DEV).to(dtype)
        q, k, v = (x.view(tokens, -1, dim) for x in qkv.split([heads * dim, kv_heads * dim, kv_heads * dim], 1))
    else:
        q, k, v = (torch.randn(tokens, h, dim, generator=g, device=DEV).to(dtype) for h in (heads, kv_heads, kv_heads))
    pages = -(-tokens // page) + 1
    pools = [torch.randn(pages, kv_heads, page, dim, generator=g, device=DEV).to(BF16) for _ in range(2)]
    before = [f64(x) for x in pools]
    slots = rng.permutation(pages * page)[:tokens]
    positions = rng.integers(0, far, tokens)
    if pad:
        positions[-pad:] = -1 - np.arange(pad)
    freq = w.rope_frequencies(rotary, base)
    weights = [(torch.rand(dim, generator=g, device=DEV) + 0.5 - offset).to(wdtype) for _ in range(2)] if norm else [None] * 2
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    p = w.params(heads, kv_heads, dim, page_size=page)
    status = w.new_status(DEV)
    q_out = torch.full((tokens, heads, dim), 7.0, dtype=BF16, device=DEV)
    k_out = torch.full((tokens, kv_heads, dim), 7.0, dtype=BF16, device=DEV)
    rope = w.Rope.from_frequencies(freq, interleaved=interleaved, factor=factor, device=DEV)
    got = w.qk_norm_rope(p, rope, q, k, v, torch.tensor(positions, dtype=torch.int32, device=DEV),
                         slots=torch.tensor(slots, device=DEV), cache=w.PagedCache(*pools, table, table[0]),
                         q_weight=weights[0], k_weight=weights[1], eps=eps, weight_offset=offset, q_out=q_out,
                         k_out=k_out, status=status)
    assert got[0] is q_out and got[1] is k_out
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    live = tokens - pad
    for out, x, wt, n in ((q_out, q, weights[0], "q"), (k_out, k, weights[1], "k")):
        _check(out[:live], x[:live], positions[:live], freq, wt, offset, eps, interleaved, factor, n)
        assert (out[live:] == 7.0).all()
    for pool, old, new, n in zip(pools, before, (f64(k_out), f64(v.to(BF16))), ("k_pool", "v_pool")):
        want = old.copy()
        for t in range(live):
            want[slots[t] // page, :, slots[t] % page] = new[t]
        assert np.array_equal(f64(pool), want), n


@pytest.mark.parametrize("dim,rotary", [(8, 2), (8, 8), (16, 6), (64, 64), (64, 14), (64, 0), (80, 80), (96, 50), (128, 128),
                                        (128, 36), (256, 64), (256, 256), (256, 250), (256, 2), (248, 126)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_dims(cuda_device, dim, rotary, interleaved):
    _run(dim + rotary, 5, 3, 2, dim, rotary, interleaved=interleaved, factor=1.25)


@pytest.mark.parametrize("kw", [
    dict(norm=False),
    dict(offset=1.0),
    dict(eps=0.25),
    dict(dtype=F32),
    dict(dtype=F32, packed=True),
    dict(wdtype=BF16),
    dict(packed=True, pad=3),
    dict(far=(1 << 31) - 1),
    dict(page=256, pad=1),
    dict(factor=-0.5),
])
@pytest.mark.parametrize("dim,rotary,interleaved", [(64, 64, False), (256, 96, True), (80, 26, False)])
def test_options(cuda_device, kw, dim, rotary, interleaved):
    _run(7, 37, 6, 2, dim, rotary, interleaved=interleaved, **kw)


@pytest.mark.parametrize("tokens,heads,kv_heads,dim", [(1, 1, 1, 64), (1, 16, 2, 256), (2, 5, 5, 80), (1537, 4, 1, 64),
                                                       (700, 24, 3, 128), (2049, 6, 2, 256), (9001, 2, 1, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes(cuda_device, tokens, heads, kv_heads, dim, interleaved):
    _run(tokens, tokens, heads, kv_heads, dim, dim // 2, packed=True, interleaved=interleaved, pad=tokens // 9)


def _small(tokens=6, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    q, k, v = (torch.randn(tokens, h, 64, generator=g, device=DEV).to(BF16) for h in (4, 2, 2))
    return w.params(4, 2, 64, page_size=16), q, k, v, torch.arange(tokens, dtype=torch.int32, device=DEV)


def test_slots_outside_the_pool_write_nothing(cuda_device):
    p, q, k, v, positions = _small()
    pools = [torch.zeros(3, 2, 16, 64, dtype=BF16, device=DEV) for _ in range(2)]
    whole = [torch.cat([torch.full_like(x, 9.0), x, torch.full_like(x, 9.0)]) for x in pools]
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    cache = w.PagedCache(whole[0][3:6], whole[1][3:6], table, table[0])
    status = w.new_status(DEV)
    slots = torch.tensor([-1, 47, 48, -2, 1 << 40, -(1 << 40)], device=DEV)
    rope = w.Rope.from_frequencies(w.rope_frequencies(64), device=DEV)
    q1, _ = w.qk_norm_rope(p, rope, q, k, v, positions, slots=slots, cache=cache, status=status)
    assert int(status.item()) == L.DEV_PAGE_OOB
    for x, new in zip(whole, (None, v)):
        assert (x[:3] == 9.0).all() and (x[6:] == 9.0).all()
        assert (x[3:6].transpose(1, 2).reshape(48, 2, 64)[:47] == 0).all()
        if new is not None:
            assert torch.equal(x[5, :, 15], new[1])
    q2, k2 = w.qk_norm_rope(p, rope, q, k, None, positions)  # every query is encoded all the same
    assert torch.equal(q1, q2) and torch.equal(whole[0][5, :, 15], k2[1])


def test_offsets_beyond_32_bits(cuda_device):
    p, q, k, v, positions = _small()
    p = w.params(4, 2, 64, page_size=256)
    pages = 70000  # 2.3e9 elements a pool
    pools = [torch.zeros(pages, 2, 256, 64, dtype=BF16, device=DEV) for _ in range(2)]
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    slots = torch.tensor([0, 255, pages * 256 - 1, pages * 256 - 256, 33333 * 256 + 7, 65535 * 256], device=DEV)
    status = w.new_status(DEV)
    _, ko = w.qk_norm_rope(p, None, q, k, v, positions, slots=slots, cache=w.PagedCache(*pools, table, table[0]),
                           k_out=torch.empty(6, 2, 64, dtype=BF16, device=DEV), status=status)
    assert int(status.item()) == 0 and torch.equal(ko, k)
    for pool, new in zip(pools, (k, v)):
        assert torch.equal(pool[slots // 256, :, slots % 256], new)
        assert int(pool.count_nonzero()) == int(new.count_nonzero())


def test_queries_or_keys_alone_in_place_and_verify_blocks(cuda_device):
    p, q, k, v, positions = _small()
    rope = w.Rope.from_frequencies(w.rope_frequencies(32), interleaved=True, device=DEV)
    q1, k1 = w.qk_norm_rope(p, rope, q, k, None, positions)
    assert w.qk_norm_rope(p, rope, q, None, None, positions)[1] is None
    assert torch.equal(w.qk_norm_rope(p, rope, q, None, None, positions)[0], q1)
    none, k2 = w.qk_norm_rope(p, rope, None, k, None, positions)
    assert none is None and torch.equal(k1, k2)
    q4, k4 = w.qk_norm_rope(p, rope, q.view(2, 3, 4, 64), k.view(2, 3, 2, 64), None, positions.view(2, 3))
    assert q4.shape == (2, 3, 4, 64) and torch.equal(q4.view_as(q1), q1) and torch.equal(k4.view_as(k1), k1)
    back = q.clone()
    w.qk_norm_rope(p, rope, back, None, None, positions, q_out=back)
    assert torch.equal(back, q1)
    assert torch.equal(w.qk_norm_rope(p, None, q, None, None, positions)[0], q)  # nothing to do: a copy
    empty, _ = w.qk_norm_rope(p, rope, q[:0], None, None, positions[:0])
    assert empty.shape == (0, 4, 64)


def test_infinities_and_nan_stay_in_their_head(cuda_device):
    p, q, k, v, positions = _small()
    rope = w.Rope.from_frequencies(w.rope_frequencies(64), device=DEV)
    good = w.qk_norm_rope(p, rope, q, None, None, positions, q_weight=torch.ones(64, device=DEV))[0]
    q[2, 1, 5] = float("nan")
    q[3, 0, 7] = float("inf")
    bad = w.qk_norm_rope(p, rope, q, None, None, positions, q_weight=torch.ones(64, device=DEV))[0]
    assert bad[2, 1].isnan().all() and bad[3, 0].isnan().any()
    good[2, 1] = bad[2, 1] = good[3, 0] = bad[3, 0] = 0
    assert torch.equal(good, bad)


def test_broadcast_heads_and_tokens(cuda_device):
    p, q, k, v, positions = _small()
    rope = w.Rope.from_frequencies(w.rope_frequencies(64), device=DEV)
    one = q[:, :1].expand(6, 4, 64)
    assert torch.equal(w.qk_norm_rope(p, rope, one, None, None, positions)[0],
                       w.qk_norm_rope(p, rope, one.contiguous(), None, None, positions)[0])
    row = q[:1].expand(6, 4, 64)
    assert torch.equal(w.qk_norm_rope(p, rope, row, None, None, positions)[0],
                       w.qk_norm_rope(p, rope, row.contiguous(), None, None, positions)[0])


def test_refusals(cuda_device):
    p, q, k, v, positions = _small()
    rope = w.Rope.from_frequencies(w.rope_frequencies(64), device=DEV)
    pools = [torch.zeros(3, 2, 16, 64, dtype=BF16, device=DEV) for _ in range(2)]
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    cache = w.PagedCache(*pools, table, table[0])
    slots = torch.arange(6, device=DEV)
    for err, args, kw in [
        (TypeError, (q.half(), k.half(), None, positions), {}),
        (TypeError, (q, k.float(), None, positions), {}),
        (ValueError, (q, k[:, :1], None, positions), {}),
        (ValueError, (q[..., ::2], k, None, positions), {}),
        (ValueError, (q, k, None, positions[:5]), {}),
        (TypeError, (q, k, None, positions.long()), {}),
        (ValueError, (q, k, v, positions), dict(slots=slots)),
        (TypeError, (q, k, v, positions), dict(slots=slots.int(), cache=cache)),
        (ValueError, (q, k, None, positions), dict(q_weight=torch.ones(32, device=DEV))),
        (TypeError, (q, k, None, positions), dict(q_weight=torch.ones(64, device=DEV, dtype=torch.half))),
        (TypeError, (q, k, None, positions), dict(q_weight=torch.ones(64, device=DEV),
                                                  k_weight=torch.ones(64, device=DEV, dtype=BF16))),
        (ValueError, (q, k, None, positions), dict(q_out=torch.empty(6, 3, 64, dtype=BF16, device=DEV))),
        (w.WmtpError, (q, k, v, positions), {}),
        (w.WmtpError, (q, k, None, positions), dict(eps=-1.0)),
        (ValueError, (q.cpu(), k, None, positions), {}),
    ]:
        with pytest.raises(err):
            w.qk_norm_rope(p, rope, *args, **kw)
    odd = torch.zeros(6 * 4 * 64 + 1, dtype=BF16, device=DEV)[1:].view(6, 4, 64)
    with pytest.raises(w.WmtpError):
        w.qk_norm_rope(p, rope, odd, None, None, positions)  # not 16-byte aligned
    with pytest.raises(ValueError):
        w.qk_norm_rope(w.params(4, 2, 64, page_size=32), rope, q, k, v, positions, slots=slots, cache=cache)
