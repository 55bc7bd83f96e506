"""A whole speculative step on the device: pages for the verify block, encoded
queries and keys into the cache, the verify attention, acceptance, the rejected
tokens' pages and ring entries taken back.  Checked against the oracle, and
captured: a replayed graph does what the eager calls do."""

import numpy as np
import pytest
import torch

import oracle
import speculative_decode_draft_b200 as w
from speculative_decode_draft_b200 import _lib as L
from _helpers import assert_close, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, GAMMA, Hq, Hkv, D, P, V = 3, 3, 16, 2, 256, 16, 517
N = GAMMA + 1
FREQ = w.rope_frequencies(64, 1e6, scaling="yarn", stretch=4.0, original=64)


class Step:
    """One layer and its state; ``__call__`` is one step on inputs that are rewritten in place."""

    def __init__(self, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.g = g
        self.p = w.params(Hq, Hkv, D, page_size=P, sinks=2, window=12, gamma_max=N)
        self.rope = w.Rope.from_frequencies(FREQ, factor=1.1, device=DEV)
        pages = 24
        pools = [torch.randn(pages, Hkv, P, D, generator=g, device=DEV).bfloat16() for _ in range(2)]
        self.pool = w.DevicePages.allocate(pages, DEV)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.cache = w.PagedCache(*pools, torch.full((B, 8), -1, dtype=torch.int32, device=DEV), self.kv_len)
        self.ring = w.Ring.allocate(self.p, B, DEV)
        self.weight = torch.rand(D, generator=g, device=DEV) + 0.5
        self.head = torch.randn(Hq * D, V, generator=g, device=DEV) * 0.08
        self.status = w.new_status(DEV)
        self.n_new = torch.full((B,), N, dtype=torch.int32, device=DEV)
        self.qkv = torch.empty(B * N, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device=DEV)
        self.tokens = torch.empty(B, GAMMA, dtype=torch.int32, device=DEV)
        self.uniforms = torch.empty(B, N, device=DEV)
        self.draw()
        # a prompt: 33, 5 and 16 tokens, not encoded (the cache holds random values already)
        w.pages_resize(self.p, self.pool, self.cache.page_table, self.kv_len,
                       torch.tensor([33, 5, 16], dtype=torch.int32, device=DEV), status=self.status)
        kv = torch.randn(B, 33, Hkv, D, generator=g, device=DEV).bfloat16()
        w.ring_append(self.p, self.ring, kv, kv, self.kv_len.clone(), status=self.status)

    def draw(self):
        g = self.g
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g, device=DEV))
        self.tokens.copy_(torch.randint(0, V, self.tokens.shape, generator=g, device=DEV))
        self.uniforms.copy_(torch.rand(self.uniforms.shape, generator=g, device=DEV) ** 8)  # some small: accepted

    def __call__(self):
        p, cache = self.p, self.cache
        base = self.kv_len.clone()
        m = w.pages_resize(p, self.pool, cache.page_table, self.kv_len, base + N, max_tokens=B * N, status=self.status)
        q, k, v = (x.view(B * N, -1, D) for x in self.qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        k_out = torch.empty(B * N, Hkv, D, dtype=torch.bfloat16, device=DEV)
        qe, _ = w.qk_norm_rope(p, self.rope, q, k, v, m.positions, slots=m.slots, cache=cache, q_weight=self.weight,
                               k_weight=self.weight, k_out=k_out, status=self.status)
        o, lse = w.verify_attn(p, qe.view(B, N, Hq, D), cache, status=self.status)
        pools = [x.clone() for x in (cache.k_pool, cache.v_pool, cache.page_table, self.kv_len)]
        w.ring_append(p, self.ring, k_out.view(B, N, Hkv, D), v.contiguous().view(B, N, Hkv, D), self.n_new, speculative=True,
                      status=self.status)
        logits = o.view(B, N, Hq * D) @ self.head
        r = w.accept_draft(logits, self.tokens, self.uniforms, status=self.status)
        lp = w.token_logprobs(logits.view(B * N, V), r.tokens.view(B * N, 1), top_k=3, status=self.status)
        w.pages_resize(p, self.pool, cache.page_table, self.kv_len, base + r.count, status=self.status)
        w.ring_append(p, self.ring, None, None, None, truncate_to=base + r.count, status=self.status)
        return dict(base=base, m=m, qe=qe, k_out=k_out, o=o, logits=logits, r=r, lp=lp, pools=pools)

    def state(self):
        return [self.cache.k_pool, self.cache.v_pool, self.cache.page_table, self.kv_len, self.pool.free, self.pool.count,
                self.ring.k, self.ring.v, self.ring.tags, self.ring.len, self.ring.committed]


def test_steps_against_the_oracle(cuda_device):
    s = Step(1)
    model = oracle.PageModel(P, 24, s.cache.page_table.tolist(), s.kv_len.tolist(), s.pool.free[: int(s.pool.count)].tolist())
    emitted = []
    for _ in range(4):
        s.draw()
        a = s()
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        base = a["base"].tolist()
        cu, positions, slots, wrong = model.resize([n + N for n in base], B * N)
        assert not wrong and a["m"].positions.tolist() == positions and a["m"].slots.tolist() == slots
        assert a["m"].cu_tokens.tolist() == cu
        wt = f64(s.weight)
        q, k, v = (f64(x.view(B * N, -1, D)) for x in s.qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        for got, x in ((a["qe"], q), (a["k_out"], k)):
            ref = oracle.rotate_heads(x, positions, FREQ, factor=1.1, weight=wt)
            size = 1.1 * np.abs(oracle.rotate_heads(x, positions, [], weight=wt)).max(-1, keepdims=True) * 2
            assert (np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * size).all()
        kp, vp, table, lens = a["pools"]
        flat = kp.transpose(1, 2).reshape(-1, Hkv, D), vp.transpose(1, 2).reshape(-1, Hkv, D)
        assert torch.equal(flat[0][slots], a["k_out"]) and np.array_equal(f64(flat[1][slots]), v)
        ref, _ = oracle.verify_attn(f64(a["qe"]).reshape(B, N, Hq, D), f64(kp), f64(vp), table.cpu().numpy(),
                                    lens.cpu().numpy(), P, 1 / np.sqrt(D))
        assert_close(f64(a["o"]), ref, "verify")
        for b in range(B):
            ids, lps, margin = oracle.accept_sequence(f64(a["logits"][b]), s.tokens[b].tolist(), f64(s.uniforms[b]))
            assert margin > 1e-5 and a["r"].tokens[b].tolist() == ids + [-1] * (N - len(ids))
            assert int(a["r"].count[b]) == len(ids)
            assert np.allclose(f64(a["r"].logprobs[b])[: len(ids)], lps, rtol=0, atol=1e-5)
            emitted.append(len(ids))
        said = a["r"].tokens.view(-1) >= 0
        assert torch.allclose(a["lp"].logprobs.view(-1)[said], a["r"].logprobs.view(-1)[said], rtol=0, atol=1e-5)
        counts = a["r"].count.tolist()
        model.resize([n + c for n, c in zip(base, counts)])
        assert s.cache.page_table.tolist() == model.table and s.kv_len.tolist() == model.kv_len
        assert s.pool.free[: int(s.pool.count)].tolist() == model.free
        assert s.ring.len.tolist() == s.ring.committed.tolist() == model.kv_len
    assert 1 in emitted and max(emitted) > 1


def test_captured_step_replays_as_eager(cuda_device):
    eager, s = Step(2), Step(2)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # the first calls come before the capture; their effect is undone
        before = [x.clone() for x in s.state()]
        s()
        for x, old in zip(s.state(), before):
            x.copy_(old)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = s()
    for x, old in zip(s.state(), before):
        x.copy_(old)
    for _ in range(5):
        eager.draw()
        for n in ("qkv", "tokens", "uniforms"):
            getattr(s, n).copy_(getattr(eager, n))
        g.replay()
        b = eager()
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0 and int(eager.status.item()) == 0
        for x, y in zip(s.state(), eager.state()):
            assert torch.equal(x, y)
        for x, y in ((a["r"], b["r"]), (a["lp"], b["lp"]), (a["m"], b["m"])):
            for n in vars(x):
                assert torch.equal(getattr(x, n), getattr(y, n)), n


def _logit_calls(seed, rows=24, vocab=60001):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g, device=DEV).bfloat16()
    ids = torch.randint(0, vocab, (rows, 2), generator=g, device=DEV).int()
    drafts = torch.randint(0, vocab, (rows // 4, 3), generator=g, device=DEV).int()
    u = torch.rand(rows // 4, 4, generator=g, device=DEV)
    q = torch.randn(rows // 4, 3, vocab, generator=g, device=DEV).bfloat16()

    def call(**kw):
        a = w.token_logprobs(x, ids, top_k=20, **kw)
        b = w.accept_draft(x.view(rows // 4, 4, vocab), drafts, u, draft_logits=q, **kw)
        return [a.logprobs, a.entropy, a.top_logprobs, a.top_ids, b.tokens, b.count, b.logprobs]
    return call


def test_two_streams_at_once(cuda_device):
    calls = [_logit_calls(i) for i in range(2)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(calls[i](stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(r, want[i]))


def test_two_captured_graphs_at_once(cuda_device):
    calls = [_logit_calls(10 + i) for i in range(2)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for x in outs[0] + outs[1]:
            x.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(x, y) for x, y in zip(outs[i], want[i]))


def test_long_chain_of_dependent_calls(cuda_device):
    """Each call reads what the one before wrote: none may start on old values."""
    p = w.params(4, 1, 64, page_size=16)
    pool = w.DevicePages.allocate(300, DEV)
    table = torch.full((7, 40), -1, dtype=torch.int32, device=DEV)
    n = torch.zeros(7, dtype=torch.int32, device=DEV)
    model = oracle.PageModel(16, 300, table.tolist(), n.tolist(), pool.free.tolist())
    rng = np.random.default_rng(5)
    status = w.new_status(DEV)
    maps = []
    plan = [rng.integers(0, 400, 7) for _ in range(60)]
    new = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in plan]
    for x in new:
        maps.append(w.pages_resize(p, pool, table, n, x, max_tokens=3000, status=status))
    for x, m in zip(plan, maps):
        cu, positions, slots, wrong = model.resize(x, 3000)
        assert not wrong and m.cu_tokens.tolist() == cu and m.slots.tolist() == slots and m.positions.tolist() == positions
    assert table.tolist() == model.table and int(status.item()) == 0


def test_refuses_a_stream_of_another_device(cuda_device):
    class Elsewhere:
        device = torch.device("cuda:7")
        cuda_stream = 0
    x = torch.zeros(1, 8, device=DEV)
    with pytest.raises(ValueError):
        w.token_logprobs(x, torch.zeros(1, 1, dtype=torch.int32, device=DEV), stream=Elsewhere())
    assert L.DEV_POOL == 0x40
