"""Timed cases of the work around the attention of one speculative decode step.

Four operators: the per-head norm and position rotation of queries and keys with the write into the
paged cache ("rope"), page tables and slot maps from request lengths ("pages"), log probabilities of
given tokens with entropy and top alternatives ("logprobs"), and the acceptance of drafted tokens
("accept").  `own` chooses between their plain torch form and the library's calls.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
NEG_INF = float("-inf")


# ---------------------------------------------------------------- cases
def _rope(name, tokens, heads, kv_heads, dim, rotary, page, far, interleaved=False, scaling="none", norm=True,
          offset=0.0, dtype="bf16", packed=True, pad=0):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "page": page, "far": far, "interleaved": interleaved, "scaling": scaling,
            "norm": norm, "offset": offset, "dtype": dtype, "packed": packed, "pad": pad}


def listed():
    return [
        # one sequence's verify block at a 1M context: 4 tokens, a quarter of the head rotated
        _rope("rope_verify_b1", 4, 16, 2, 256, 64, 64, 1 << 20, scaling="yarn", offset=1.0),
        # 64 sequences drafting one token each, fp32 projections, whole head rotated in pairs, some lanes idle
        _rope("rope_draft_b64", 64, 4, 1, 64, 64, 16, 1 << 17, interleaved=True, dtype="fp32", pad=7),
        # a ragged chunk of prompt tokens, no norm, linear position scaling, separate q, k and v
        _rope("rope_chunk_odd", 1537, 16, 2, 256, 96, 64, 1 << 18, scaling="linear", norm=False, packed=False, pad=3),
        # a prompt of 32K tokens written at once
        _rope("rope_prompt_32k", 32768, 16, 2, 256, 256, 64, 1 << 15, scaling="bands"),
        # 4 sequences at up to 1M tokens growing by a verify block and taking it back
        {"name": "pages_verify_b4", "op": "pages", "batch": 4, "page": 64, "context": 1 << 20, "grow": 4,
         "shrink": 0, "short": False},
        # 512 requests of a full server: prompt chunks arrive while others finish, the pool runs out
        {"name": "pages_prompts_b512", "op": "pages", "batch": 512, "page": 16, "context": 1 << 15, "grow": 2048,
         "shrink": 5, "short": True},
        # the verify block of one sequence
        {"name": "logprobs_b1", "op": "logprobs", "rows": 4, "vocab": 131072, "dtype": "bf16", "given": 1, "top": 5,
         "temperature": False, "masked": False, "slack": 0},
        # 36 rows of an odd vocabulary under a token mask, at each row's temperature
        {"name": "logprobs_odd_masked", "op": "logprobs", "rows": 36, "vocab": 129281, "dtype": "fp32", "given": 3,
         "top": 20, "temperature": True, "masked": True, "slack": 31},
        # a prompt's tokens scored
        {"name": "logprobs_score_1k", "op": "logprobs", "rows": 1024, "vocab": 131072, "dtype": "bf16", "given": 1,
         "top": 8, "temperature": False, "masked": False, "slack": 0},
        # one sequence, three drafted tokens that carry no distribution
        {"name": "accept_b1_g3", "op": "accept", "batch": 1, "gamma": 3, "vocab": 131072, "dtype": "bf16",
         "drafted": False, "greedy": 0, "ragged": False},
        # 32 sequences with the drafts' logits, some of them greedy, of different draft lengths
        {"name": "accept_b32_g5", "op": "accept", "batch": 32, "gamma": 5, "vocab": 129281, "dtype": "bf16",
         "drafted": True, "greedy": 4, "ragged": True},
        # fp32 logits of 16 sequences and eight drafts
        {"name": "accept_b16_g8", "op": "accept", "batch": 16, "gamma": 8, "vocab": 50257, "dtype": "fp32",
         "drafted": True, "greedy": 0, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "pages", "logprobs", "accept"])
    if op == "rope":
        heads, kv, dim = rng.choice([(16, 2, 256), (4, 1, 64), (8, 8, 64), (24, 3, 128), (5, 5, 80), (6, 2, 256)])
        most = (32768 * 20 * 256) // ((heads + 2 * kv) * dim * 2)
        c = _rope("", _log(rng, 1, most), heads, kv, dim, 2 * rng.randint(1, dim // 2), rng.choice([16, 32, 64, 128, 256]),
                  _log(rng, 1 << 12, 1 << 22), rng.random() < 0.5, rng.choice(["none", "linear", "yarn", "bands"]),
                  rng.random() < 0.7, rng.choice([0.0, 1.0]), rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.6)
        c["pad"] = rng.choice([0, 0, rng.randint(1, 9)]) if c["tokens"] > 1 else 0
    elif op == "pages":
        batch = _log(rng, 1, 1024)
        page = rng.choice([16, 32, 64, 128, 256])
        c = {"name": "", "op": "pages", "batch": batch, "page": page, "context": _log(rng, 64, (1 << 24) // batch),
             "grow": _log(rng, 1, max(2, min(8192, (1 << 20) // batch))), "shrink": rng.choice([0, 2, 7]),
             "short": rng.random() < 0.3}
    elif op == "logprobs":
        vocab = _log(rng, 512, 262144)
        c = {"name": "", "op": "logprobs", "rows": _log(rng, 1, min(4096, (1024 * 131072) // (2 * vocab))), "vocab": vocab,
             "dtype": rng.choice(["bf16", "fp16", "fp32"]), "given": rng.randint(1, 9), "top": rng.choice([0, 1, 5, 20, 32, 64]),
             "temperature": rng.random() < 0.5, "masked": rng.random() < 0.4, "slack": rng.choice([0, 0, rng.randint(1, 64)])}
    else:
        vocab = _log(rng, 512, 262144)
        gamma = rng.randint(1, 8)
        c = {"name": "", "op": "accept", "batch": _log(rng, 1, max(1, min(64, (32 * 6 * 129281) // ((gamma + 1) * vocab)))),
             "gamma": gamma, "vocab": vocab, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "drafted": rng.random() < 0.6,
             "greedy": rng.choice([0, 1, 3]), "ragged": rng.random() < 0.5}
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _frequencies(rotary, scaling):
    """(angle per position of each pair, factor on the rotated values), as Python floats."""
    base = 1e7 if scaling in ("none", "yarn") else 5e5
    freq = [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    if scaling == "linear":
        return [f / 8.0 for f in freq], 1.0
    if scaling == "yarn":  # pairs that turn rarely in 32K positions are slowed by 4, fast ones kept, a ramp between
        def dim(turns):
            return rotary * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rotary - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(rotary // 2)]
        return [f / 4.0 * r + f * (1.0 - r) for f, r in zip(freq, ramp)], 0.1 * math.log(4.0) + 1.0
    if scaling == "bands":  # the same by the turns that a pair makes in 8192 positions: below 1 slowed by 8, above 4 kept
        keep = [min(max((8192 * f / (2 * math.pi) - 1.0) / 3.0, 0.0), 1.0) for f in freq]
        return [f / 8.0 * (1.0 - s) + f * s for f, s in zip(freq, keep)], 1.0
    return freq, 1.0


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _prepare_rope(c, g):
    T, Hq, Hkv, D, P = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    dt = DTYPES[c["dtype"]]
    if c["packed"]:  # one projection's output, cut into q, k and v
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=DEV).mul_(1.5).to(dt)
        q, k, v = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).mul_(1.5).to(dt) for h in (Hq, Hkv, Hkv))
    pages = -(-T // P) + 2
    place = torch.randperm((pages - 1) * P, generator=g, device=DEV)[:T]  # the last page stays out of use
    positions = torch.randint(0, c["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
    if c["pad"]:  # rows behind the last token of a padded batch
        positions[-c["pad"]:] = -1
        place[-c["pad"]:] = -1
    weights = [torch.rand(D, generator=g, device=DEV) + 0.5 - c["offset"] for _ in range(2)] if c["norm"] else [None, None]
    freq, factor = _frequencies(c["rotary"], c["scaling"])
    s = {"q": q, "k": k, "v": v, "positions": positions, "slots": place, "qw": weights[0], "kw": weights[1],
         "k_pool": torch.randn(pages, Hkv, P, D, generator=g, device=DEV).to(torch.bfloat16),
         "v_pool": torch.randn(pages, Hkv, P, D, generator=g, device=DEV).to(torch.bfloat16),
         "q_out": torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV),
         "freq": torch.tensor(freq, dtype=torch.float64, device=DEV), "factor": factor}
    if own:  # the handles that a program keeps for all its calls
        import speculative_decode_draft_b200 as w
        s["p"] = w.params(Hq, Hkv, D, page_size=P)
        s["rope"] = w.Rope.from_frequencies(freq, interleaved=c["interleaved"], factor=factor, device=DEV)
        table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
        s["cache"] = w.PagedCache(s["k_pool"], s["v_pool"], table, table[0])
    return s


def _prepare_pages(c, g):
    B, P = c["batch"], c["page"]
    width = -(-(c["context"] + c["grow"]) // P)
    kv_len = torch.randint(1, c["context"] + 1, (B,), generator=g, device=DEV)
    new_len = kv_len + torch.randint(1, c["grow"] + 1, (B,), generator=g, device=DEV)
    if c["grow"] <= 16:  # a decode step: every sequence grows by the same block
        new_len = kv_len + c["grow"]
    if c["shrink"]:  # these requests take back a part, or all where it is little
        less = torch.randint(0, c["grow"] + 1, (B,), generator=g, device=DEV)
        new_len = torch.where(torch.arange(B, device=DEV) % c["shrink"] == 1, (kv_len - less).clamp_(min=0), new_len)
    held = (kv_len + P - 1) // P
    mine = torch.arange(width, device=DEV)[None, :] < held[:, None]
    used = int(mine.sum())
    need = int(((new_len + P - 1) // P - held).clamp_(min=0).sum())
    pages = B * width + 1
    spare = need // 3 if c["short"] else min(need + 5, pages - used)
    order = torch.randperm(pages, generator=g, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int64, device=DEV)
    table[mine] = order[:used]
    free = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    free[:spare] = order[used:used + spare].int()
    most = B * c["grow"] + 3
    return {"kv_len": kv_len.int(), "old_len": kv_len.int().clone(), "new_len": new_len.int(), "table": table.int(), "free": free,
            "count": torch.tensor([spare], dtype=torch.int32, device=DEV), "tokens": most, "page": P, "pages": pages}


def _logits(shape, g, dtype, sharp):
    """Logits with a few likely tokens over a broad rest."""
    x = torch.randn(shape, generator=g, device=DEV).mul_(2.0)
    likely = torch.randint(0, shape[-1], (*shape[:-1], 6), generator=g, device=DEV)
    up = torch.rand((*shape[:-1], 6), generator=g, device=DEV).mul_(sharp).add_(6.0)
    return x.scatter_reduce_(-1, likely, up, "amax").to(dtype)  # a column drawn twice: the larger, whatever the order


def _prepare_logprobs(c, g):
    R, V = c["rows"], c["vocab"]
    x = _logits((R, V + c["slack"]), g, DTYPES[c["dtype"]], 8.0)
    tokens = torch.randint(0, V, (R, c["given"]), generator=g, device=DEV)
    tokens[:, 0] = x[:, :V].argmax(-1)
    if c["masked"]:  # a grammar leaves some tokens: few, or most
        left = torch.where(torch.arange(R, device=DEV) % 3 == 0, 20.0 / V, 0.7)
        for a in range(0, R, 256):
            b = min(R, a + 256)
            x[a:b, :V].masked_fill_(torch.rand(b - a, V, generator=g, device=DEV) > left[a:b, None], NEG_INF)
        x.scatter_(1, torch.randint(0, V, (R, 1), generator=g, device=DEV), 3.0)
    x[:, V:] = float("nan")  # columns behind the vocabulary hold anything
    temperature = torch.rand(R, generator=g, device=DEV) * 1.5 + 0.25 if c["temperature"] else None
    return {"x": x[:, :V], "tokens": tokens.int(), "temperature": temperature}


def _prepare_accept(c, g):
    B, G, V = c["batch"], c["gamma"], c["vocab"]
    dt = DTYPES[c["dtype"]]
    target = _logits((B, G + 1, V), g, dt, 8.0)
    draft = (target[:, :G].float() + torch.randn(B, G, V, generator=g, device=DEV) * 0.5).to(dt)
    noise = torch.rand(B, G, V, generator=g, device=DEV).clamp_(1e-12).log_().neg_().log_().neg_()
    tokens = (draft.float() + noise).argmax(-1).int() if c["drafted"] else draft.argmax(-1).int()
    temperature = torch.rand(B, generator=g, device=DEV) + 0.5
    if c["greedy"]:
        temperature[torch.arange(B, device=DEV) % c["greedy"] == 0] = 0.0
    num = torch.randint(0, G + 1, (B,), generator=g, device=DEV, dtype=torch.int32) if c["ragged"] else None
    return {"target": target, "draft": draft if c["drafted"] else None, "tokens": tokens, "num": num,
            "uniforms": torch.rand(B, G + 1, generator=g, device=DEV), "temperature": temperature}


_PREPARE = {"rope": _prepare_rope, "pages": _prepare_pages, "logprobs": _prepare_logprobs, "accept": _prepare_accept}


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed))
    s["case"] = case
    if own and case["op"] == "pages":
        import speculative_decode_draft_b200 as w
        s["p"] = w.params(16, 2, 256, page_size=case["page"])
        s["pool"] = w.DevicePages(s["free"], s["count"])
    return s


# ---------------------------------------------------------------- plain forms
def _rotate_plain(x, cos, sin, rotary, interleaved):
    turn, rest = x[..., :rotary], x[..., rotary:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turn[..., : rotary // 2], turn[..., rotary // 2:]
        turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turn, rest], -1)


def _norm_plain(x, weight, offset, eps):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * (weight + offset)


def _rope_plain(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    q, k = (_rotate_plain(_norm_plain(s[n], s[n + "w"], c["offset"], 1e-6), cos, sin, c["rotary"], c["interleaved"])
            .to(torch.bfloat16) for n in "qk")
    there = s["positions"] >= 0
    s["q_out"].copy_(torch.where(there[:, None, None], q, s["q_out"]))
    P, last = c["page"], s["k_pool"].shape[0] * c["page"] - 1
    slot = torch.where(there & (s["slots"] >= 0), s["slots"], last)  # rows without a slot put back what the last one holds
    page, row = slot // P, slot % P
    stays = (slot == last)[:, None, None]
    for pool, new in ((s["k_pool"], k), (s["v_pool"], s["v"].to(torch.bfloat16))):
        pool[page, :, row] = torch.where(stays, pool[page, :, row], new)
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _resize_plain(s, new_len, most):
    P, table = s["page"], s["table"].long()
    B, width = table.shape
    old, new, count = s["kv_len"].long(), new_len.long(), s["count"].long()
    valid = (old >= 0) & (old <= width * P) & (new >= 0) & (new <= width * P)
    hold, want = (old + P - 1) // P, (new + P - 1) // P
    released = ((hold - want).clamp(min=0) * valid).sum()
    tokens = (new - old).clamp(min=0) * valid
    fits = ((want - hold).clamp(min=0) * valid).cumsum(0) <= count + released
    served = valid & ((tokens == 0) | (fits & (tokens.cumsum(0) <= most)))
    tokens = tokens * served
    j = torch.arange(width, device=DEV)[None, :]
    gives = (j >= want[:, None]) & (j < hold[:, None]) & served[:, None]
    takes = (j >= hold[:, None]) & (j < want[:, None]) & served[:, None]
    rank = gives.flatten().long().cumsum(0).view(B, width) - 1
    stack = torch.cat([s["free"].long(), s["free"].new_zeros(1).long()])
    stack[torch.where(gives, count + released - 1 - rank, s["pages"])] = table
    at = count + released - takes.flatten().long().cumsum(0).view(B, width)
    table = torch.where(takes, stack[torch.where(takes, at, 0)], torch.where(gives, -1, table))
    lens = torch.where(served, new, old)
    end = tokens.cumsum(0)
    t = torch.arange(most, device=DEV)
    b = torch.searchsorted(end, t, right=True).clamp(max=B - 1)
    position = old[b] + t - (end - tokens)[b]
    live = t < end[-1]
    position = torch.where(live, position, 0)
    slot = table[b, position // P] * P + position % P
    s["table"].copy_(table)
    s["kv_len"].copy_(lens)
    s["free"].copy_(stack[:-1])
    s["count"].copy_(count + released - takes.sum())
    cu = torch.cat([end.new_zeros(1), end]).int()
    return {"cu": cu, "positions": torch.where(live, position, -1).int(), "slots": torch.where(live, slot, -1)}


def _pages_plain(s):
    first = _resize_plain(s, s["new_len"], s["tokens"])
    back = _resize_plain(s, s["old_len"], s["tokens"])
    return {"there": first, "back": back, "table": s["table"], "kv_len": s["kv_len"], "free": s["free"], "count": s["count"]}


def _ordered(x):
    """Whole numbers in the order of x: larger values first, then lower columns."""
    bits = (x.float() + 0.0).view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    return (bits << 32) - torch.arange(x.shape[-1], device=x.device)


def _logprobs_plain(s):
    c, x = s["case"], s["x"].float()
    scale = torch.ones((), device=DEV) if s["temperature"] is None else (1.0 / s["temperature"])[:, None]
    top = x.max(-1, keepdim=True).values
    y = (x - top) * scale
    e = torch.exp(y)
    total = e.sum(-1, keepdim=True)
    log_total = total.log()
    entropy = log_total - torch.where(e > 0, e * y, 0.0).sum(-1, keepdim=True) / total
    out = {"logprobs": torch.gather(y, 1, s["tokens"].long()) - log_total, "entropy": entropy[:, 0],
           "lse": (top * scale + log_total)[:, 0]}
    if c["top"]:
        ids = _ordered(x).topk(c["top"], -1).indices
        values = torch.gather(y, 1, ids) - log_total
        out["top_logprobs"] = values
        out["top_ids"] = torch.where(values == NEG_INF, -1, ids).int()
    return out


def _accept_plain(s):
    x = s["target"].double()
    B, n, V = x.shape
    greedy = s["temperature"] == 0
    t = torch.where(greedy, 1.0, s["temperature"].double())[:, None, None]
    logp = (x - x.max(-1, keepdim=True).values) / t
    logp = logp - logp.exp().sum(-1, keepdim=True).log()
    p = logp.exp()
    d = s["tokens"].long()
    if s["draft"] is None:
        q = torch.zeros_like(p[:, :-1]).scatter_(-1, d[..., None], 1.0)
    else:
        y = s["draft"].double()
        y = (y - y.max(-1, keepdim=True).values) / t
        q = y.exp() / y.exp().sum(-1, keepdim=True)
    num = torch.full((B,), n - 1, device=DEV) if s["num"] is None else s["num"].long()
    best = torch.where(x == x.max(-1, keepdim=True).values, torch.arange(V, device=DEV), V).min(-1).values
    pd, qd = (torch.gather(v[:, : n - 1], 2, d[..., None])[..., 0] for v in (p, q))
    u = s["uniforms"].double()
    kept = torch.where(greedy[:, None], best[:, :-1] == d, u[:, :-1] * qd < pd)
    kept = kept & (torch.arange(n - 1, device=DEV) < num[:, None])
    kept = kept.long().cumprod(1).sum(1)
    at = torch.arange(B, device=DEV)
    rest = p[at, kept]
    minus = torch.where((kept < num)[:, None], q[at, kept.clamp(max=n - 2)], 0.0)
    left = (rest - minus).clamp(min=0)
    weight = torch.where(left.sum(-1, keepdim=True) > 0, left, rest)
    mass = weight.cumsum(-1)
    final = torch.searchsorted(mass, u[:, -1:] * mass[:, -1:], right=True)[:, 0].clamp(max=V - 1)
    final = torch.where(greedy, best[at, kept], final)
    i = torch.arange(n, device=DEV)[None, :]
    padded = torch.cat([d, d[:, :1]], 1)
    tokens = torch.where(i < kept[:, None], padded, torch.where(i == kept[:, None], final[:, None], -1))
    said = torch.gather(logp, 2, tokens.clamp(min=0)[..., None])[..., 0]
    return {"tokens": tokens.int(), "count": (kept + 1).int(), "logprobs": torch.where(tokens < 0, 0.0, said).float()}


_PLAIN = {"rope": _rope_plain, "pages": _pages_plain, "logprobs": _logprobs_plain, "accept": _accept_plain}


# ---------------------------------------------------------------- the library's calls
def _rope_own(s):
    import speculative_decode_draft_b200 as w
    w.qk_norm_rope(s["p"], s["rope"], s["q"], s["k"], s["v"], s["positions"], slots=s["slots"], cache=s["cache"],
                   q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, weight_offset=s["case"]["offset"], q_out=s["q_out"])
    return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _pages_own(s):
    import speculative_decode_draft_b200 as w
    a = w.pages_resize(s["p"], s["pool"], s["table"], s["kv_len"], s["new_len"], max_tokens=s["tokens"])
    b = w.pages_resize(s["p"], s["pool"], s["table"], s["kv_len"], s["old_len"], max_tokens=s["tokens"])
    there, back = ({"cu": m.cu_tokens, "positions": m.positions, "slots": m.slots} for m in (a, b))
    return {"there": there, "back": back, "table": s["table"], "kv_len": s["kv_len"], "free": s["free"], "count": s["count"]}


def _logprobs_own(s):
    import speculative_decode_draft_b200 as w
    r = w.token_logprobs(s["x"], s["tokens"], top_k=s["case"]["top"], temperature=s["temperature"])
    out = {"logprobs": r.logprobs, "entropy": r.entropy, "lse": r.lse}
    if s["case"]["top"]:
        out["top_logprobs"], out["top_ids"] = r.top_logprobs, r.top_ids
    return out


def _accept_own(s):
    import speculative_decode_draft_b200 as w
    r = w.accept_draft(s["target"], s["tokens"], s["uniforms"], draft_logits=s["draft"], num_draft=s["num"],
                       temperature=s["temperature"])
    return {"tokens": r.tokens, "count": r.count, "logprobs": r.logprobs}


_OWN = {"rope": _rope_own, "pages": _pages_own, "logprobs": _logprobs_own, "accept": _accept_own}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- floors
def work(case):
    c = case
    if c["op"] == "rope":
        T, D, b = c["tokens"] - c["pad"], c["dim"], BYTES[c["dtype"]]
        rows = c["heads"] + 2 * c["kv_heads"]
        return {"bytes": T * rows * D * (b + 2) + 12 * c["tokens"],
                "flops": T * (c["heads"] + c["kv_heads"]) * (3 * c["rotary"] + (4 * D if c["norm"] else 0))}
    if c["op"] == "pages":
        tokens = c["batch"] * (c["grow"] if c["grow"] <= 16 else c["grow"] / 2)
        moved = tokens / c["page"]
        return {"bytes": 2 * (12 * tokens + 8 * moved + 16 * c["batch"]), "flops": 8 * tokens}
    if c["op"] == "logprobs":
        n = c["rows"] * c["vocab"]
        return {"bytes": n * BYTES[c["dtype"]] + c["rows"] * (8 * c["given"] + 8 * c["top"] + 8), "flops": 6 * n}
    rows = c["batch"] * (c["gamma"] + 1 + (c["gamma"] if c["drafted"] else 0))
    return {"bytes": rows * c["vocab"] * BYTES[c["dtype"]] + 16 * c["batch"] * (c["gamma"] + 1), "flops": 4 * rows * c["vocab"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _rope_exact(c, s):
    T, D, rot = c["tokens"], c["dim"], c["rotary"]
    out = {}
    pair = torch.arange(rot // 2, device=DEV)
    first = 2 * pair if c["interleaved"] else pair
    second = first + (1 if c["interleaved"] else rot // 2)
    angle = s["positions"].double()[:, None, None] * s["freq"][None, None, :]
    for n in "qk":
        x = s[n].double().clone()
        if c["norm"]:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / D + 1e-6) * (s[n + "w"].double() + c["offset"])
        z = torch.polar(torch.full_like(angle, s["factor"]), angle) * torch.complex(x[..., first], x[..., second])
        x[..., first], x[..., second] = z.real, z.imag
        out[n] = x
    live = (s["positions"] >= 0).nonzero()[:, 0]
    q = torch.zeros_like(out["q"])
    q[live] = out["q"][live]
    pools = {}
    for n, new in (("k_pool", out["k"]), ("v_pool", s["v"].double())):
        flat = s[n].double().transpose(1, 2).reshape(-1, c["kv_heads"], D).contiguous()
        flat[s["slots"][live]] = new[live]
        pools[n] = flat.view(-1, c["page"], c["kv_heads"], D).transpose(1, 2).contiguous()
    return {"q": q, **pools}


def _logprobs_exact(c, s):
    parts = []
    for r in range(0, c["rows"], 64):
        x = s["x"][r:r + 64].double()
        if s["temperature"] is not None:
            x = x / s["temperature"][r:r + 64, None].double()
        lse = torch.logsumexp(x, -1, keepdim=True)
        lp = x - lse
        ent = -torch.where(x == NEG_INF, 0.0, lp.exp() * lp).sum(-1)
        got = [lp.gather(1, s["tokens"][r:r + 64].long()), ent, lse[:, 0]]
        if c["top"]:
            got.append(lp.topk(c["top"], -1).values)
        parts.append(got)
    got = [torch.cat(v) for v in zip(*parts)]
    out = {"logprobs": got[0], "entropy": got[1], "lse": got[2]}
    if c["top"]:
        out["top_logprobs"], out["top_ids"] = got[3], None
    return out


def _accept_exact(c, s):
    B, G = c["batch"], c["gamma"]
    temps = s["temperature"].tolist()
    drafts, coins = s["tokens"].tolist(), s["uniforms"].double().tolist()
    nums = [G] * B if s["num"] is None else s["num"].tolist()
    said = torch.zeros(B, G + 1, dtype=torch.float64)
    for b in range(B):
        t = temps[b] or 1.0
        p = torch.softmax(s["target"][b].double() / t, -1)
        q = None if s["draft"] is None else torch.softmax(s["draft"][b].double() / t, -1)
        k = 0
        while k < nums[b]:
            d = drafts[b][k]
            if temps[b] == 0:
                ok = int(s["target"][b, k].double().argmax()) == d or float(s["target"][b, k].max()) == float(s["target"][b, k, d])
                ok = ok and int((s["target"][b, k] == s["target"][b, k].max()).nonzero()[0]) == d
            else:
                ok = coins[b][k] * (1.0 if q is None else float(q[k, d])) < float(p[k, d])
            if not ok:
                break
            said[b, k] = p[k, d].log()
            k += 1
        w = p[k].clone()
        if k < nums[b]:
            if q is None:
                w[drafts[b][k]] = 0.0
            else:
                w = (w - q[k]).clamp(min=0)
        if temps[b] == 0:
            final = int((s["target"][b, k] == s["target"][b, k].max()).nonzero()[0])
        else:
            mass = w.cumsum(0)
            final = int((mass > coins[b][G] * mass[-1]).nonzero()[0])
        said[b, k] = p[k, final].log()
    return {"tokens": None, "count": None, "logprobs": said}


def exact(case, seed):
    if case["op"] == "pages":
        return None
    s = _PREPARE[case["op"]](case, _gen(seed))
    return {"rope": _rope_exact, "logprobs": _logprobs_exact, "accept": _accept_exact}[case["op"]](case, s)
