"""pages_resize against the Python page model: every table, stack, length and
slot equal."""

from ctypes import byref, c_size_t

import numpy as np
import pytest
import torch

import oracle
import speculative_decode_draft_b200 as w
from speculative_decode_draft_b200 import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BITS = {"len": L.DEV_LEN_OOB, "pool": L.DEV_POOL, "page": L.DEV_PAGE_OOB}


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Both:
    """The device state and the model, started alike."""

    def __init__(self, seed, batch, width, page, pages, lens):
        rng = np.random.default_rng(seed)
        order = rng.permutation(pages)
        table = np.full((batch, width), -1)
        n = 0
        for b in range(batch):
            h = -(-lens[b] // page)
            table[b, :h] = order[n:n + h]
            n += h
        self.p = w.params(16, 2, 256, page_size=page)
        self.model = oracle.PageModel(page, pages, table, lens, order[n:])
        free = np.full(pages, -1)
        free[: pages - n] = order[n:]
        self.pool = w.DevicePages(_i32(free), _i32([pages - n]))
        self.table, self.len = _i32(table).view(batch, width), _i32(lens)

    def resize(self, new, most):
        status = w.new_status(DEV)
        m = w.pages_resize(self.p, self.pool, self.table, self.len, _i32(new), max_tokens=most, status=status)
        cu, positions, slots, wrong = self.model.resize(new, most)
        assert int(status.item()) == sum(BITS[x] for x in wrong)
        assert self.table.tolist() == self.model.table and self.len.tolist() == self.model.kv_len
        count = int(self.pool.count.item())
        assert count == len(self.model.free) and self.pool.free[:count].tolist() == self.model.free
        if most:
            assert m.cu_tokens.tolist() == cu and m.positions.tolist() == positions and m.slots.tolist() == slots
        else:
            assert m is None
        return wrong


@pytest.mark.parametrize("batch,width,page,pages", [(1, 1, 16, 1), (1, 9, 16, 9), (3, 5, 32, 11), (7, 40, 64, 200),
                                                    (33, 6, 256, 150), (1025, 7, 16, 5000), (2500, 3, 128, 6000)])
@pytest.mark.parametrize("most", [0, 40, 100000])
def test_random_lengths(cuda_device, batch, width, page, pages, most):
    rng = np.random.default_rng(batch)
    s = Both(batch, batch, width, page, pages, [0] * batch)
    cap, seen = width * page, set()
    for step in range(8):
        kind = step % 4
        if kind == 0:
            new = rng.integers(0, cap + 1, batch)
        elif kind == 1:  # a decode step
            new = np.array(s.model.kv_len) + rng.integers(0, 6, batch)
        elif kind == 2:  # half of them end or shrink
            new = np.where(rng.random(batch) < 0.5, rng.integers(0, cap + 1, batch) // 3, s.model.kv_len)
        else:
            new = rng.integers(-2, cap + 3, batch)
        seen |= s.resize(new, most)
    assert "len" in seen or batch < 100


def test_long_rows_and_many_pages(cuda_device):
    width, page = 16384, 64  # 2^20 tokens
    s = Both(5, 4, width, page, 50000, [1000000, 1, 700001, 0])
    s.resize([1 << 20, 64, 0, 640], 1 << 17)
    s.resize([1000000, 60, 900000, 0], 0)
    s.resize([1000001, 61, 900001, 300000], 300003)
    s.resize([0, 0, 0, 0], 5)


def test_growth_taken_back(cuda_device):
    s = Both(6, 9, 30, 16, 300, [100] * 9)
    table, free = s.table.clone(), s.pool.free.clone()
    s.resize([400] * 9, 2700)
    s.resize([100] * 9, 0)
    assert torch.equal(table, s.table) and torch.equal(free, s.pool.free)


def test_first_that_does_not_fit_stops_growth_not_release(cuda_device):
    s = Both(7, 4, 10, 16, 12, [16, 160, 0, 16])  # all 12 pages held
    assert s.resize([33, 160, 0, 16], 100) == {"pool"}
    assert s.resize([33, 32, 1, 32], 100) == set()  # 8 come back, 2 + 1 + 1 go
    assert s.resize([34, 33, 160, 33], 100) == {"pool"}  # the third needs 9: the fourth waits too
    assert s.resize([34, 33, 1, 33], 1) == set()  # one token on a page that is still free, one row of the map
    assert s.resize([35, 34, 1, 33], 1) == {"pool"}  # two tokens for a map of one row


def test_inconsistent_state(cuda_device):
    for count in (-1, 13, 5):  # negative, more than there are, and more once pages come back
        s = Both(8, 2, 4, 16, 6, [16, 64])
        s.pool.count[:] = count
        before = [x.clone() for x in (s.table, s.len, s.pool.free, s.pool.count)]
        status = w.new_status(DEV)
        m = w.pages_resize(s.p, s.pool, s.table, s.len, _i32([20, 0]), max_tokens=50, status=status)
        assert int(status.item()) == L.DEV_POOL
        assert all(torch.equal(a, b) for a, b in zip(before, (s.table, s.len, s.pool.free, s.pool.count)))
        assert (m.cu_tokens == 0).all() and (m.slots == -1).all() and (m.positions == -1).all()
    s = Both(9, 2, 4, 16, 8, [20, 20])
    s.table[0, 1] = 99  # a page that is not there
    s.table[1, 1] = -5
    status = w.new_status(DEV)
    m = w.pages_resize(s.p, s.pool, s.table, s.len, _i32([22, 3]), max_tokens=4, status=status)
    assert int(status.item()) == L.DEV_PAGE_OOB
    assert m.slots.tolist() == [-1] * 4 and m.positions.tolist() == [20, 21, -1, -1]


def test_map_in_buffers_of_any_alignment(cuda_device):
    """Through the C ABI: positions and slots need the alignment of their elements only."""
    lib, B, most = w.load(), 40, 5003
    p = w.params(16, 2, 256, page_size=32)
    pool = w.DevicePages.allocate(400, DEV)
    model = oracle.PageModel(32, 400, [[-1] * 9] * B, [0] * B, pool.free.tolist())
    table, kv_len = _i32(np.full((B, 9), -1)), _i32([0] * B)
    new = np.random.default_rng(3).integers(0, 200, B)
    cu = torch.empty(B + 1, dtype=torch.int32, device=DEV)
    positions = torch.full((most + 2,), 7, dtype=torch.int32, device=DEV)
    slots = torch.full((most + 2,), 7, dtype=torch.int64, device=DEV)
    size = c_size_t(0)
    new_len = _i32(new)
    args = (byref(p), B, table.data_ptr(), 9, kv_len.data_ptr(), new_len.data_ptr())
    out = (cu.data_ptr(), positions.data_ptr() + 4, slots.data_ptr() + 8, most)
    assert lib.wmtp_pages_resize(*args, None, None, 400, *out, None, byref(size), None, None) == 0
    ws = torch.empty(size.value, dtype=torch.uint8, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    assert lib.wmtp_pages_resize(*args, pool.free.data_ptr(), pool.count.data_ptr(), 400, *out, ws.data_ptr(), byref(size),
                                 None, st) == 0
    want = model.resize(new, most)
    assert cu.tolist() == want[0] and positions.tolist() == [7] + want[1] + [7] and slots.tolist() == [7] + want[2] + [7]
    assert kv_len.tolist() == model.kv_len and table.tolist() == model.table


def test_empty_batch(cuda_device):
    p = w.params(16, 2, 256)
    pool = w.DevicePages.allocate(4, DEV)
    m = w.pages_resize(p, pool, _i32(np.zeros((0, 3))), _i32([]), _i32([]), max_tokens=3)
    assert m.cu_tokens.tolist() == [0] and m.slots.tolist() == [-1] * 3
    assert w.pages_resize(p, pool, _i32(np.zeros((0, 3))), _i32([]), _i32([])) is None


def test_refusals(cuda_device):
    p, pool, table, n = w.params(16, 2, 256), w.DevicePages.allocate(4, DEV), _i32([[-1, -1]]), _i32([0])
    for err, args, kw in [
        (ValueError, (table[0], n, n), {}),
        (ValueError, (table, _i32([0, 0]), n), {}),
        (TypeError, (table, n, n.long()), {}),
        (TypeError, (table.long(), n, n), {}),
        (ValueError, (table, n, n), dict(max_tokens=-1)),
        (ValueError, (_i32([[-1, -1, 0]])[:, ::2], n, n), {}),
        (ValueError, (table, n.cpu(), n), {}),
    ]:
        with pytest.raises(err):
            w.pages_resize(p, pool, *args, **kw)
    with pytest.raises(w.WmtpError):
        w.pages_resize(w.params(16, 2, 256, page_size=24), pool, table, n, n)
    with pytest.raises(ValueError):
        w.pages_resize(p, w.DevicePages(pool.free, n.repeat(2)), table, n, n)
