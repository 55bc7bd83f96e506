"""Host-only checks of include/wmtp_step.h: arguments are refused before the
GPU is touched.  The pointers below are never dereferenced."""

import ctypes
from ctypes import byref, c_size_t

import pytest
import torch

import speculative_decode_draft_b200 as w
from speculative_decode_draft_b200 import _lib as L

A = 4096  # an aligned address
INVALID, UNSUPPORTED, WORKSPACE = L.WMTP_ERR_INVALID_ARG, L.WMTP_ERR_UNSUPPORTED, L.WMTP_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    from speculative_decode_draft_b200 import build
    build.build()
    return L.load()


def _rope(lib, heads=(16, 2), dim=256, page=64, rope=(A, 64, 0, 1.0), tokens=4, dtype=0, q=(A, 4096, 256),
          k=(A, 512, 256), v=(A, 512, 256), positions=A, slots=A, kv=(A, A, 8), qw=None, kw=None, wt=0, offset=0.0,
          eps=1e-6, q_out=A, k_out=None):
    p = w.params(*heads, dim, page_size=page)
    r = None if rope is None else L.RopeDesc(*rope)
    desc = None if kv is None else L.PagedKVDesc(kv[0], kv[1], kv[2], None, 0, None)
    return lib.wmtp_qk_norm_rope(byref(p), None if r is None else byref(r), tokens, dtype, *q, *k, *v, positions,
                                 slots, None if desc is None else byref(desc), qw, kw, wt, offset, eps, q_out, k_out,
                                 None, None)


NONE = (None, 0, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVALID),
    (dict(heads=(0, 2)), INVALID),
    (dict(heads=(16, 0)), INVALID),
    (dict(heads=(70000, 2)), UNSUPPORTED),
    (dict(dim=0), UNSUPPORTED),
    (dict(dim=60), UNSUPPORTED),
    (dict(dim=264), UNSUPPORTED),
    (dict(dtype=1), UNSUPPORTED),  # fp16
    (dict(dtype=7), UNSUPPORTED),
    (dict(wt=1), UNSUPPORTED),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(offset=float("inf")), INVALID),
    (dict(rope=(A, 63, 0, 1.0)), INVALID),
    (dict(rope=(A, 258, 0, 1.0)), INVALID),
    (dict(rope=(A, -2, 0, 1.0)), INVALID),
    (dict(rope=(None, 64, 0, 1.0)), INVALID),
    (dict(rope=(A + 4, 64, 0, 1.0)), INVALID),
    (dict(rope=(A, 64, 0, float("nan"))), INVALID),
    (dict(q=NONE), INVALID),  # with a q_out
    (dict(q_out=None), INVALID),
    (dict(q=NONE, q_out=None, k=NONE, v=NONE, slots=None), INVALID),
    (dict(k=NONE), INVALID),  # slots without keys
    (dict(slots=None, v=NONE), INVALID),  # keys with no place to go
    (dict(slots=None, k_out=A), INVALID),  # values with no place to go
    (dict(v=NONE), INVALID),
    (dict(k=NONE, v=NONE, slots=None, k_out=A), INVALID),
    (dict(page=48), UNSUPPORTED),
    (dict(kv=None), INVALID),
    (dict(kv=(None, A, 8)), INVALID),
    (dict(kv=(A, None, 8)), INVALID),
    (dict(kv=(A, A, 0)), INVALID),
    (dict(kv=(A + 8, A, 8)), INVALID),
    (dict(slots=A + 4), INVALID),
    (dict(positions=None), INVALID),
    (dict(positions=A + 2), INVALID),
    (dict(q=(A + 2, 4096, 256)), INVALID),
    (dict(q=(A, 4100, 256)), INVALID),
    (dict(k=(A, 512, 260)), INVALID),
    (dict(v=(A, -512, 256)), INVALID),
    (dict(qw=A + 8), INVALID),
    (dict(q_out=A + 8), INVALID),
    (dict(k_out=A + 8), INVALID),
])
def test_qk_norm_rope_refuses(lib, kw, code):
    assert _rope(lib, **kw) == code


def test_qk_norm_rope_without_tokens_is_a_noop(lib):
    assert _rope(lib, tokens=0, positions=None) == 0


def _pages(lib, page=64, batch=2, table=A, width=8, kv_len=A, new_len=A, free=A, count=A, pages=8, cu=A, pos=A,
           slots=A, most=16, ws=A, size=1 << 20):
    p = w.params(16, 2, 256, page_size=page)
    have = c_size_t(size)
    code = lib.wmtp_pages_resize(byref(p), batch, table, width, kv_len, new_len, free, count, pages, cu, pos, slots,
                                 most, ws, byref(have), None, None)
    return code if ws is not None or free is not None else (code, have.value)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID),
    (dict(batch=65536), UNSUPPORTED),
    (dict(page=24), UNSUPPORTED),
    (dict(width=0), INVALID),
    (dict(width=1 << 25), UNSUPPORTED),  # 2^31 tokens
    (dict(pages=0), INVALID),
    (dict(most=-1), INVALID),
    (dict(most=0), INVALID),  # a map without rows
    (dict(cu=None), INVALID),
    (dict(pos=None), INVALID),
    (dict(slots=None), INVALID),
    (dict(free=None), INVALID),
    (dict(count=None), INVALID),
    (dict(table=None), INVALID),
    (dict(kv_len=None), INVALID),
    (dict(new_len=None), INVALID),
    (dict(slots=A + 4), INVALID),
    (dict(table=A + 2), INVALID),
    (dict(ws=A + 16), WORKSPACE),
    (dict(batch=500, size=8), WORKSPACE),
    (dict(batch=500, ws=None), WORKSPACE),
    (dict(most=100000, ws=None), WORKSPACE),
])
def test_pages_resize_refuses(lib, kw, code):
    assert _pages(lib, **kw) == code


def test_pages_resize_of_nothing_is_a_noop(lib):
    assert _pages(lib, batch=0, table=None, kv_len=None, new_len=None, cu=None, pos=None, slots=None, most=0) == 0
    assert _pages(lib, ws=None, free=None) == (0, 0)  # few sequences need no scratch
    assert _pages(lib, ws=None, free=None, batch=33)[1] > 0


def _logprobs(lib, rows=2, vocab=100, dtype=0, logits=A, stride=100, temperature=None, tokens=A, n=1, k=4, lp=A,
              ent=A, lse=A, top=A, ids=A):
    return lib.wmtp_token_logprobs(rows, vocab, dtype, logits, stride, temperature, tokens, n, k, lp, ent, lse, top,
                                   ids, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID),
    (dict(vocab=0), INVALID),
    (dict(vocab=(1 << 30) + 1, rows=1), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED),
    (dict(k=65), UNSUPPORTED),
    (dict(k=-1), INVALID),
    (dict(n=-1), INVALID),
    (dict(stride=99), INVALID),
    (dict(logits=None), INVALID),
    (dict(logits=A + 1), INVALID),
    (dict(dtype=2, logits=A + 2), INVALID),
    (dict(tokens=None), INVALID),
    (dict(lp=None), INVALID),
    (dict(top=None), INVALID),
    (dict(ids=None), INVALID),
    (dict(tokens=A + 2), INVALID),
    (dict(temperature=A + 2), INVALID),
])
def test_token_logprobs_refuses(lib, kw, code):
    assert _logprobs(lib, **kw) == code


def test_token_logprobs_without_rows_is_a_noop(lib):
    assert _logprobs(lib, rows=0, logits=None, tokens=None, lp=None) == 0


def _accept(lib, batch=2, n=4, vocab=100, dtype=0, target=(A, 400, 100), draft=(A, 300, 100), tokens=A, uniforms=A,
            num=None, temperature=None, out=A, count=A, lp=A, ws=A, size=1 << 20):
    have = c_size_t(size)
    code = lib.wmtp_accept_draft(batch, n, vocab, dtype, *target, *draft, tokens, uniforms, num, temperature, out,
                                 count, lp, ws, byref(have), None, None)
    return code, have.value


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID),
    (dict(batch=65536), UNSUPPORTED),
    (dict(n=0), INVALID),
    (dict(n=33), UNSUPPORTED),
    (dict(vocab=0), INVALID),
    (dict(dtype=5), UNSUPPORTED),
    (dict(ws=A + 16), WORKSPACE),
    (dict(size=8), WORKSPACE),
    (dict(target=(None, 400, 100)), INVALID),
    (dict(target=(A + 1, 400, 100)), INVALID),
    (dict(target=(A, -400, 100)), INVALID),
    (dict(draft=(A + 1, 300, 100)), INVALID),
    (dict(tokens=None), INVALID),
    (dict(uniforms=None), INVALID),
    (dict(uniforms=A + 2), INVALID),
    (dict(out=None), INVALID),
    (dict(count=None), INVALID),
])
def test_accept_draft_refuses(lib, kw, code):
    assert _accept(lib, **kw)[0] == code


def test_accept_draft_sizes(lib):
    code, size = _accept(lib, ws=None)
    assert code == 0 and size > 0
    assert _accept(lib, batch=0, ws=None) == (0, 0)
    assert _accept(lib, batch=0)[0] == 0
    have = ctypes.c_void_p(None)
    assert lib.wmtp_accept_draft(1, 2, 8, 0, None, 0, 0, None, 0, 0, None, None, None, None, None, None, None, None,
                                 ctypes.cast(have, ctypes.POINTER(c_size_t)), None, None) == INVALID


def test_wrappers_refuse_cpu_tensors():
    p = w.params(4, 1, 64)
    x = torch.zeros(2, 8)
    i = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        w.token_logprobs(x, i)
    with pytest.raises(ValueError, match="CUDA"):
        w.accept_draft(x[None], i[None, :, 0], x[None, :, 0])
    with pytest.raises(ValueError, match="CUDA"):
        w.pages_resize(p, w.DevicePages.allocate(4, "cpu"), i, i[:, 0], i[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        w.qk_norm_rope(p, None, x.view(1, 2, 8), None, None, i[:1, 0])
    with pytest.raises(ValueError):
        w.qk_norm_rope(p, None, None, None, None, i[:, 0])


def test_wrappers_refuse_what_is_no_tensor_or_no_params():
    x = torch.zeros(2, 8)
    i = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(TypeError, match="logits"):
        w.token_logprobs([[0.0]], i)
    with pytest.raises((TypeError, ValueError)):
        w.accept_draft(x[None], i[None, :, 0], None)
    with pytest.raises(TypeError):
        w.pages_resize(7, w.DevicePages.allocate(4, "cpu"), i, i[:, 0], i[:, 0])
    with pytest.raises(TypeError, match="params"):
        w.pages_resize(b"1234", w.DevicePages.allocate(4, "cpu"), i, i[:, 0], i[:, 0])
    with pytest.raises(AttributeError):
        w.pages_resize(w.params(4, 1, 64), None, i, i[:, 0], i[:, 0])


def test_rope_turns_are_whole_turns_modulo_one():
    import math
    r = w.Rope.from_frequencies([2 * math.pi * 0.25, 2 * math.pi * 1.25, -2 * math.pi * 0.25, 0.0], device="cpu")
    turns = [t % (1 << 64) for t in r.turn.tolist()]
    assert turns[0] == turns[1] == 1 << 62 and turns[2] == 3 << 62 and turns[3] == 0
    with pytest.raises(ValueError):
        w.Rope.from_frequencies([math.inf], device="cpu")
    pages = w.DevicePages.allocate(3, "cpu")
    assert pages.free.tolist() == [2, 1, 0] and pages.count.tolist() == [3]
