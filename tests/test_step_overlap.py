"""wmtp_qk_norm_rope refuses outputs over rows that other tokens read.

Host only but for the last test: the refused calls' pointers are never dereferenced."""

from ctypes import byref

import pytest
import torch

import speculative_decode_draft_b200 as w
from speculative_decode_draft_b200 import _lib as L

Hq, Hkv, D, P, T, PAGES = 4, 2, 64, 16, 6, 3
ROW = (Hq + 2 * Hkv) * D  # elements of a packed token
AT = 1 << 30              # of the buffer in question; the others lie far from it
FAR = [(1 << 32) + (i << 28) for i in range(8)]


@pytest.fixture(scope="module")
def lib():
    from speculative_decode_draft_b200 import build
    build.build()
    return L.load()


def _call(lib, q=None, k=None, v=None, q_out=FAR[3], k_out=FAR[4], pools=(FAR[5], FAR[6]), tokens=T, dtype=L.DTYPE_BF16):
    q, k, v = q or (FAR[0], Hq * D, D), k or (FAR[1], Hkv * D, D), v or (FAR[2], Hkv * D, D)
    p = w.params(Hq, Hkv, D, page_size=P)
    kv = L.PagedKVDesc(*pools, PAGES, None, 0, None)
    return lib.wmtp_qk_norm_rope(byref(p), None, tokens, dtype, *q, *k, *v, FAR[7], FAR[7], byref(kv), None, None, 0, 0.0,
                                 1e-6, q_out, k_out, None, None)


OUT = T * Hq * D * 2   # bytes of q_out
KOUT = T * Hkv * D * 2
POOL = PAGES * Hkv * P * D * 2
PACKED = dict(q=(AT, ROW, D), k=(AT + 2 * Hq * D, ROW, D), v=(AT + 2 * (Hq + Hkv) * D, ROW, D))


@pytest.mark.parametrize("kw", [
    dict(**PACKED, q_out=AT),                                   # over the start of a packed projection
    dict(**PACKED, q_out=AT + 2 * ROW * T - 16),                # over its last values
    dict(**PACKED, q_out=AT - OUT + 16),
    dict(**PACKED, k_out=AT + 2 * Hq * D),                      # where the first token's keys are
    dict(**PACKED, k_out=AT + 2 * Hq * D, tokens=2),
    dict(q=(AT, Hq * D, D), q_out=AT + 16),                     # its own rows, shifted
    dict(q=(AT, Hq * D, D), q_out=AT - 2 * D),
    dict(q=(AT, Hq * D, D), q_out=AT, dtype=L.DTYPE_FP32),      # rows of another size
    dict(q=(AT, D, T * D), q_out=AT),                           # heads first
    dict(q=(AT, 0, D), q_out=AT),                               # one token for all
    dict(q=(AT, Hq * D, 0), q_out=AT),                          # one head for all
    dict(k=(AT, Hkv * D, D), q_out=AT),
    dict(v=(AT, Hkv * D, D), q_out=AT + KOUT - 16),
    dict(q=(AT, Hq * D, D), k_out=AT),
    dict(k=(AT, Hkv * D, D), k_out=AT + 2 * D),
    dict(v=(AT, Hkv * D, D), k_out=AT),
    dict(q_out=AT, k_out=AT + OUT - 16),
    dict(q_out=AT, k_out=AT),
    dict(q_out=AT, pools=(AT + OUT - 16, FAR[6])),
    dict(k_out=AT + POOL - 16, pools=(FAR[5], AT)),
    dict(pools=(AT, AT)),
    dict(pools=(AT, AT + POOL - 16)),
])
def test_overlapping_buffers_are_refused(lib, kw):
    assert _call(lib, **kw) == L.WMTP_ERR_INVALID_ARG


@pytest.mark.gpu
def test_outputs_that_take_the_place_of_their_own_rows_or_touch(cuda_device):
    """In place where that is sound, next to the inputs, and in the gaps between a view's rows."""
    g = torch.Generator(device="cuda:0")
    g.manual_seed(1)
    p = w.params(Hq, Hkv, D, page_size=P)
    rope = w.Rope.from_frequencies(w.rope_frequencies(D), device="cuda:0")
    bf16 = dict(dtype=torch.bfloat16, device="cuda:0")
    positions = torch.arange(3, 3 + T, dtype=torch.int32, device="cuda:0")
    q, k = (torch.randn(T, h, D, generator=g, device="cuda:0").bfloat16() for h in (Hq, Hkv))
    want_q, want_k = w.qk_norm_rope(p, rope, q, k, None, positions)
    a, b = q.clone(), k.clone()
    w.qk_norm_rope(p, rope, a, b, None, positions, q_out=a, k_out=b)
    assert torch.equal(a, want_q) and torch.equal(b, want_k)
    # one token of a packed projection: its queries and keys are contiguous
    packed = torch.cat([q[:1].flatten(), k[:1].flatten()])
    a, b = packed[: Hq * D].view(1, Hq, D), packed[Hq * D:].view(1, Hkv, D)
    w.qk_norm_rope(p, rope, a, b, None, positions[:1], q_out=a, k_out=b)
    assert torch.equal(a, want_q[:1]) and torch.equal(b, want_k[:1])
    # next to one another
    room = torch.empty(T * (2 * Hq + 2 * Hkv) * D, **bf16)
    a, b, c, d = (x.view(T, -1, D) for x in room.split([T * Hq * D, T * Hq * D, T * Hkv * D, T * Hkv * D]))
    a.copy_(q), c.copy_(k)
    w.qk_norm_rope(p, rope, a, c, None, positions, q_out=b, k_out=d)
    assert torch.equal(a, q) and torch.equal(b, want_q) and torch.equal(c, k) and torch.equal(d, want_k)
    # between two tokens' rows
    room = torch.empty(2, 3 * Hq * D, **bf16)
    a, b = room[:, : Hq * D].view(2, Hq, D), room[0, Hq * D:].view(2, Hq, D)
    a.copy_(q[:2])
    w.qk_norm_rope(p, rope, a, None, None, positions[:2], q_out=b)
    assert torch.equal(a, q[:2]) and torch.equal(b, want_q[:2])
    # a packed projection written over
    packed = torch.randn(T, ROW, generator=g, device="cuda:0").bfloat16()
    a, b, _ = (x.view(T, -1, D) for x in packed.split([Hq * D, Hkv * D, Hkv * D], 1))
    over = packed.view(-1)[: T * Hq * D].view(T, Hq, D)
    with pytest.raises(w.WmtpError):
        w.qk_norm_rope(p, rope, a, b, None, positions, q_out=over)
