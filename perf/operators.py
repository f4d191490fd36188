"""What the serving and training operators around the paged cache are measured on.

Four operators: rotary positions (with their gradient, and fused with the write
into a paged cache), attention of a tree of drafted tokens over a paged cache
(with the move of the accepted tokens' rows), single-token decode that
accumulates every cached token's attention weight, and the eviction of the
tokens of least weight.  ``run`` computes them in elementary torch operations, or
with ``own`` through this package's entry points.
"""
import math
import random

import torch

own = False

HEADS = ((64, 8, 64), (32, 8, 128), (8, 1, 64), (12, 12, 64), (16, 4, 128))  # query heads, KV heads, head dim


# ---------------------------------------------------------------------------
# Cases.


def listed():
    return [
        # A training step's rotation of queries and keys and of their gradients: 2 sequences of 8192 tokens.
        dict(name="rope_train", op="rope", tokens=16384, hq=64, hkv=8, d=64, rotary=64, interleaved=False,
             scaling="none", far=8192, grad=True),
        # One decode step of 64 requests: the new tokens' queries rotated, their keys rotated into the cache.
        dict(name="rope_append_decode", op="append", batch=64, len_lo=1, len_hi=4096, new_lo=1, new_hi=1, hq=64,
             hkv=8, d=64, page=16, rotary=64, interleaved=False, scaling="yarn", lens=1),
        # Chunked prefill of 8 requests, half of each 128-wide head rotated, interleaved pairs.
        dict(name="rope_append_extend", op="append", batch=8, len_lo=0, len_hi=4096, new_lo=512, new_hi=8192, hq=32,
             hkv=8, d=128, page=64, rotary=64, interleaved=True, scaling="bands", lens=2),
        # One user's draft of 7 tokens checked against a short conversation: latency.
        dict(name="tree_one", op="tree", batch=1, len_lo=2000, len_hi=2000, n_lo=7, n_hi=7, hq=64, hkv=8, d=64,
             page=16, sink=True, first=0, last=0, lens=3),
        # A serving batch with drafts of 16 to 64 tokens over caches of 1k to 16k tokens.
        dict(name="tree_batch", op="tree", batch=16, len_lo=1024, len_hi=16384, n_lo=16, n_hi=64, hq=64, hkv=8, d=64,
             page=16, sink=True, first=0, last=0, lens=4),
        # Drafts over long caches of which the first 1024 and the last 7168 tokens are seen.
        dict(name="tree_window", op="tree", batch=32, len_lo=8192, len_hi=65536, n_lo=8, n_hi=32, hq=32, hkv=8, d=128,
             page=64, sink=False, first=1024, last=7168, lens=5),
        # The rows of 8 requests' accepted draft tokens moved to the end of their prefixes.
        dict(name="accept_few", op="accept", batch=8, len_lo=500, len_hi=2000, n_lo=16, n_hi=32, hkv=8, d=64, page=16,
             lens=6),
        # The same for a full batch with larger drafts, wide heads and large pages.
        dict(name="accept_batch", op="accept", batch=256, len_lo=64, len_hi=1024, n_lo=32, n_hi=64, hkv=8, d=128,
             page=64, lens=7),
        # Decode steps of 4 short requests that keep each token's accumulated weight: latency.
        dict(name="weights_few", op="weights", batch=4, len_lo=256, len_hi=2048, hq=32, hkv=8, d=128, page=64,
             sink=False, first=0, last=0, per_head=True, lens=8),
        # The same for a full serving batch of 1k to 32k tokens.
        dict(name="weights_batch", op="weights", batch=64, len_lo=1024, len_hi=32768, hq=64, hkv=8, d=64, page=16,
             sink=True, first=0, last=0, per_head=True, lens=9),
        # Two requests brought down to 1024 tokens, the same tokens for all heads.
        dict(name="evict_few", op="evict", batch=2, len_lo=1100, len_hi=3000, hkv=8, d=64, page=16, budget=1024,
             first=4, last=256, per_head=False, lens=10),
        # A batch brought down to 4096 tokens per KV head.
        dict(name="evict_batch", op="evict", batch=32, len_lo=8192, len_hi=16384, hkv=8, d=128, page=64, budget=4096,
             first=4, last=1024, per_head=True, lens=11),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "tree", "accept", "weights", "evict"))
    hq, hkv, d = rng.choice(HEADS)
    page = rng.choice((8, 16, 32, 64, 128))
    lens = rng.randrange(1 << 30)
    rotary = rng.choice((d, d, d // 2, d // 4 + 2, d - 14))
    rope = dict(rotary=rotary, interleaved=rng.random() < 0.5, scaling=rng.choice(("none", "linear", "base", "yarn", "bands")))
    window = rng.choice(((0, 0), (0, 0), (1024, 7168), (4, 509), (0, 1000)))
    if op == "rope":
        return dict(op=op, tokens=_log_int(rng, 1, 16000), hq=hq, hkv=hkv, d=d, far=_log_int(rng, 1000, 1000000),
                    grad=rng.random() < 0.6, **rope)
    if op == "append":
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4000)
        return dict(op=op, batch=_log_int(rng, 1, 64 if new == 1 else 8), len_lo=0, len_hi=_log_int(rng, 16, 4096),
                    new_lo=max(1, new // 3), new_hi=new, hq=hq, hkv=hkv, d=d, page=page, lens=lens, **rope)
    if op == "tree":
        n = _log_int(rng, 1, 64)
        hi = _log_int(rng, 64, 16000)
        return dict(op=op, batch=_log_int(rng, 1, 16), len_lo=hi // 3, len_hi=hi, n_lo=(n + 1) // 2, n_hi=n, hq=hq,
                    hkv=hkv, d=d, page=page, sink=rng.random() < 0.5, first=window[0], last=window[1], lens=lens)
    if op == "accept":
        n = _log_int(rng, 2, 64)
        hi = _log_int(rng, 16, 2000)
        return dict(op=op, batch=_log_int(rng, 1, 128), len_lo=hi // 2, len_hi=hi, n_lo=(n + 1) // 2, n_hi=n, hkv=hkv,
                    d=d, page=page, lens=lens)
    if op == "weights":
        hi = _log_int(rng, 64, 32000)
        return dict(op=op, batch=_log_int(rng, 1, 32), len_lo=max(1, hi // 8), len_hi=hi, hq=hq, hkv=hkv, d=d,
                    page=page, sink=rng.random() < 0.5, first=window[0], last=window[1], per_head=rng.random() < 0.5,
                    lens=lens)
    hi = _log_int(rng, 200, 16000)
    budget = max(16, int(hi * rng.uniform(0.2, 0.9)))
    return dict(op=op, batch=_log_int(rng, 1, 16), len_lo=hi // 2, len_hi=hi, hkv=hkv, d=d, page=page, budget=budget,
                first=rng.choice((0, 4)), last=budget // rng.choice((3, 5, 16)), per_head=rng.random() < 0.5, lens=lens)


def lengths(case):
    """(cached tokens before the new ones, new tokens) of every request, fixed by the case."""
    rng = random.Random(case["lens"])
    lo, hi = case.get("n_lo", case.get("new_lo", 0)), case.get("n_hi", case.get("new_hi", 0))
    return [(rng.randint(case["len_lo"], case["len_hi"]), rng.randint(lo, hi)) for _ in range(case["batch"])]


def frequencies(case):
    """Inverse frequencies in radians per position, and the factor on the rotated part."""
    r, base, s, old = case["rotary"], 10000.0, 8.0, 4096.0
    kind = case["scaling"]
    if kind == "base":
        base = base * s ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if kind == "linear":
        return [x / s for x in f], 1.0
    if kind == "yarn":  # pairs that turn often in the old context stay, slow ones are stretched, a ramp between
        def dim(turns):
            return r * math.log(old / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), r - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(r // 2)]
        return [x * (1 - t) + x / s * t for x, t in zip(f, ramp)], 0.1 * math.log(s) + 1.0
    if kind == "bands":  # by the number of turns in the old context: below 1 stretched, above 4 kept, blended between
        turns = [old * x / (2 * math.pi) for x in f]
        keep = [min(max((t - 1.0) / (4.0 - 1.0), 0.0), 1.0) for t in turns]
        return [x * t + x / s * (1 - t) for x, t in zip(f, keep)], 1.0
    return f, 1.0


# ---------------------------------------------------------------------------
# Inputs.


class _Gen:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda", dtype=torch.bfloat16)

    def uniform(self, *shape, dtype=torch.float32):
        return torch.rand(*shape, generator=self.g, device="cuda", dtype=dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(gen, case, total):
    """Caches and a page table for requests of `total` tokens, pages in random order."""
    page = case["page"]
    n = torch.tensor([max(1, -(-t // page)) for t in total], device="cuda")
    pool = int(n.sum())
    perm = torch.randperm(pool, generator=gen.g, device="cuda").int()
    at = torch.arange(int(n.max()), device="cuda")[None, :]
    at = at.expand(len(total), -1)
    start = (n.cumsum(0) - n)[:, None]
    table = torch.where(at < n[:, None], perm[(start + at).clamp(max=pool - 1)], -1).int().contiguous()
    return (gen.normal(pool, page, case["hkv"], case["d"]), gen.normal(pool, page, case["hkv"], case["d"]), table)


def prepare(case, seed):
    gen, op = _Gen(seed), case["op"]
    s = dict(case=case, op=op)
    if op in ("rope", "append"):
        f, s["attn_scale"] = frequencies(case)
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    if op == "rope":
        t, d = case["tokens"], case["d"]
        s["q"], s["k"] = gen.normal(t, case["hq"], d), gen.normal(t, case["hkv"], d)
        s["positions"] = torch.randint(0, case["far"], (t,), generator=gen.g, device="cuda").int()
        if case["grad"]:
            s["q"].requires_grad_(), s["k"].requires_grad_()
            s["dq"], s["dk"] = gen.normal(t, case["hq"], d), gen.normal(t, case["hkv"], d)
        return s
    lens = lengths(case)
    total = [p + n for p, n in lens]
    s["k_cache"], s["v_cache"], s["table"] = _cache(gen, case, total)
    s["seqlens"] = _i32(total)
    s["max_len"], s["max_new"] = max(total), max(n for _, n in lens)
    if op in ("append", "tree"):
        rows = sum(n for _, n in lens)
        new = torch.tensor([n for _, n in lens], device="cuda")
        s["cu"] = torch.cat([new.new_zeros(1), new.cumsum(0)]).int()
        s["q"] = gen.normal(rows, case["hq"], case["d"])
    if op == "append":
        s["k_new"], s["v_new"] = (gen.normal(rows, case["hkv"], case["d"]) for _ in range(2))
    if op in ("tree", "weights"):
        s["sink"] = gen.uniform(case["hq"]) * 6 - 2 if case["sink"] else None
    if op == "tree":  # every node hangs on an earlier one of its request or, -1, on the prefix
        row = torch.arange(rows, device="cuda")
        own_start = s["cu"].long()[torch.bucketize(row, s["cu"][1:].long(), right=True)]
        s["parents"] = ((gen.uniform(rows, dtype=torch.float64) * (row - own_start + 1)).floor() - 1).int()
    if op == "accept":  # the accepted nodes of each request, in order, behind its prefix
        most = min(8, case["n_lo"])
        s["base"] = _i32([p for p, _ in lens])
        s["counts"] = torch.randint(0, most + 1, (len(lens),), generator=gen.g, device="cuda").int()
        rank = gen.uniform(len(lens), s["max_new"])
        rank = torch.where(torch.arange(s["max_new"], device="cuda") < _i32([n for _, n in lens])[:, None], rank, 2.0)
        s["src"] = (s["base"][:, None] + rank.argsort(1)[:, :most].sort(1).values.int()).contiguous()
    if op == "weights":
        s["q"] = gen.normal(len(lens), case["hq"], case["d"])
    if op in ("weights", "evict"):
        heads = case["hkv"] if case["per_head"] else 1
        w = gen.uniform(len(lens), heads, s["max_len"]) ** 4
        w = torch.where(gen.uniform(len(lens), heads, s["max_len"]) < 0.05, 0.0, w)
        s["weights"] = torch.where(torch.arange(s["max_len"], device="cuda") < s["seqlens"][:, None, None], w, 0.0)
    if op == "evict":
        s["weights_out"] = torch.empty_like(s["weights"])
    return s


# ---------------------------------------------------------------------------
# The plain forms: 32 bits, angles in 64.


def _cos_sin(positions, inv_freq, scale):
    a = positions.double()[:, None] * inv_freq
    return (a.cos() * scale).float(), (a.sin() * scale).float()


def _rotate(x, cos, sin, interleaved):
    """x (rows, heads, d), cos / sin (rows, rotary / 2)."""
    x, h = x.float(), cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((y, x[..., 2 * h:]), -1).bfloat16()


def _new_slots(s):
    """Request and cache slot of every new row."""
    row = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.bucketize(row, s["cu"][1:].long(), right=True)
    t = s["seqlens"].long()[b] - (s["cu"].long()[b + 1] - row)
    return b, t, _slot(s, b, t)


def _slot(s, b, t):
    page = s["case"]["page"]
    return s["table"][b, t // page].long() * page + t % page


def _rows(s, name):
    """A cache as rows of tokens."""
    return s[name].view(-1, *s[name].shape[2:])


def _gathered(s, name):
    """Every request's cached tokens, padded: (batch, tokens, KV heads, d) in 32 bits."""
    b = torch.arange(s["seqlens"].numel(), device="cuda")[:, None]
    t = torch.arange(s["max_len"], device="cuda")[None, :]
    t = torch.minimum(t, s["seqlens"].long()[:, None] - 1)
    return _rows(s, name)[_slot(s, b, t)].float()


def _in_window(t, pos, case):
    """Whether a query at `pos` sees position `t`, both in the same sequence."""
    seen = t <= pos
    if case["last"] > 0:
        seen = seen & ((t < case["first"]) | (t > pos - case["last"]))
    return seen


def _softmax_parts(scores, sink):
    """(probabilities, log of the denominator); `sink` broadcasts against the rows of `scores`, or is None."""
    top = scores.amax(-1, keepdim=True)
    if sink is not None:
        top = torch.maximum(top, sink[..., None])
    e = (scores - top).exp()
    z = e.sum(-1, keepdim=True)
    if sink is not None:
        z = z + (sink[..., None] - top).exp()
    return e / z, (top + z.log()).squeeze(-1)


def _plain_rope(s):
    case = s["case"]
    cos, sin = _cos_sin(s["positions"], s["inv_freq"], s["attn_scale"])
    out = [_rotate(s[n].detach(), cos, sin, case["interleaved"]) for n in ("q", "k")]
    if case["grad"]:  # the transpose of a rotation is the rotation back
        out += [_rotate(s[n], cos, -sin, case["interleaved"]) for n in ("dq", "dk")]
    return out


def _plain_append(s):
    _, t, slot = _new_slots(s)
    cos, sin = _cos_sin(t, s["inv_freq"], s["attn_scale"])
    _rows(s, "k_cache")[slot] = _rotate(s["k_new"], cos, sin, s["case"]["interleaved"])
    _rows(s, "v_cache")[slot] = s["v_new"]
    return [_rotate(s["q"], cos, sin, s["case"]["interleaved"]), s["k_cache"], s["v_cache"]]


def _plain_tree(s):
    case, n = s["case"], s["max_new"]
    b, t, _ = _new_slots(s)
    batch, hq, hkv, d = s["seqlens"].numel(), case["hq"], case["hkv"], case["d"]
    node = torch.arange(b.numel(), device="cuda") - s["cu"].long()[b]
    # ancestors: the powers of the child-to-parent matrix (its nilpotent part is summed by (1 + P)^n)
    step = torch.zeros(batch, n, n + 1, dtype=torch.float64, device="cuda")
    step[b, node, s["parents"].long() % (n + 1)] = 1.0  # column n: the prefix
    see = torch.linalg.matrix_power(step[..., :n] + torch.eye(n, dtype=torch.float64, device="cuda"), n) > 0
    prefix = (s["seqlens"] - (s["cu"][1:] - s["cu"][:-1])).long()
    pos = prefix[:, None] + see.sum(-1) - 1  # of every node
    q = torch.zeros(batch, n, hq, d, device="cuda")
    q[b, node] = s["q"].float()
    q = q.view(batch, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    scores = q @ _gathered(s, "k_cache").permute(0, 2, 3, 1) * d ** -0.5
    # which tokens a node sees: the prefix by position, the draft by ancestry and position
    key = torch.arange(s["max_len"], device="cuda")[None, :] - prefix[:, None]  # node of the token, < 0: prefix
    key_node = key.clamp(0, n - 1)[:, None, :].expand(-1, n, -1)
    key_pos = torch.where(key < 0, key + prefix[:, None], pos.gather(1, key.clamp(0, n - 1)))
    seen = (key[:, None, :] < 0) | (see.gather(2, key_node) & (key < n)[:, None, :])
    seen = seen & _in_window(key_pos[:, None, :], pos[..., None], case)
    seen = seen & (torch.arange(s["max_len"], device="cuda") < s["seqlens"][:, None])[:, None, :]
    scores = scores.view(batch, hq, n, -1).masked_fill(~seen[:, None], -math.inf)
    scores = torch.where(torch.arange(n, device="cuda")[:, None] < (s["cu"][1:] - s["cu"][:-1])[:, None, None, None],
                         scores, 0.0)
    p, lse = _softmax_parts(scores, None if s["sink"] is None else s["sink"][:, None].expand(batch, -1, n))
    out = p.view(batch, hkv, -1, s["max_len"]) @ _gathered(s, "v_cache").transpose(1, 2)
    out = out.view(batch, hq, n, d)[b, :, node].bfloat16()
    return [out, lse[b, :, node].t().contiguous()]


def _plain_accept(s):
    src, base = s["src"].long(), s["base"].long()
    at = torch.arange(src.shape[1], device="cuda")
    keep = at < s["counts"][:, None]
    b = torch.arange(src.shape[0], device="cuda")[:, None].expand_as(src)[keep]
    from_, to = _slot(s, b, src[keep]), _slot(s, b, (base[:, None] + at)[keep])
    for name in ("k_cache", "v_cache"):
        _rows(s, name)[to] = _rows(s, name)[from_]
    return [s["k_cache"], s["v_cache"]]


def _plain_weights(s):
    case = s["case"]
    batch, hq, hkv, d = s["seqlens"].numel(), case["hq"], case["hkv"], case["d"]
    q = s["q"].float().view(batch, hkv, hq // hkv, d)
    scores = q @ _gathered(s, "k_cache").permute(0, 2, 3, 1) * d ** -0.5
    t = torch.arange(s["max_len"], device="cuda")
    seen = _in_window(t, (s["seqlens"] - 1)[:, None], case)[:, None, None]
    scores = scores.masked_fill(~seen, -math.inf)
    p, lse = _softmax_parts(scores, None if s["sink"] is None else s["sink"].view(1, hkv, -1).expand(batch, -1, -1))
    out = (p @ _gathered(s, "v_cache").transpose(1, 2)).view(batch, hq, d).bfloat16()
    s["weights"] += p.sum(2) if case["per_head"] else p.sum((1, 2))[:, None]
    return [out, lse.view(batch, hq), s["weights"]]


def _plain_evict(s):
    case, w = s["case"], s["weights"]
    batch, heads, cap = w.shape
    budget, t = case["budget"], torch.arange(cap, device="cuda")
    length = s["seqlens"].long()[:, None, None]
    key = torch.where((t < case["first"]) | (t >= length - case["last"]), math.inf, w)
    key = torch.where(t < length, key, -math.inf)
    kept = key.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    new = torch.minimum(length, length.new_tensor(budget))
    at = torch.arange(min(budget, cap), device="cuda")
    kept = torch.where(at < new, kept, cap).sort(-1).values  # ascending, the padding last
    live = kept < cap
    s["weights_out"].zero_()
    s["weights_out"][..., :at.numel()] = torch.where(live, w.gather(-1, kept.clamp(max=cap - 1)), 0.0)
    hkv = case["hkv"]
    b = torch.arange(batch, device="cuda")[:, None, None].expand(-1, hkv, at.numel())
    h = torch.arange(hkv, device="cuda")[None, :, None].expand_as(b)
    live_h, kept_h = live.expand(-1, hkv, -1), kept.expand(-1, hkv, -1)
    b, h, from_, to = b[live_h], h[live_h], kept_h[live_h], at.expand_as(kept_h)[live_h]
    from_, to = _slot(s, b, from_), _slot(s, b, to)
    for name in ("k_cache", "v_cache"):
        _rows(s, name)[to, h] = _rows(s, name)[from_, h]
    kept = torch.nn.functional.pad(torch.where(live, kept, -1), (0, budget - at.numel()), value=-1)
    return [new.view(-1).int(), kept.int(), s["weights_out"], s["k_cache"], s["v_cache"]]


# ---------------------------------------------------------------------------
# One pass.


def _own(s):
    import paged_kv_sink_gb300 as ext
    case, op = s["case"], s["op"]
    if op == "rope":
        kw = dict(interleaved=case["interleaved"], attn_scale=s["attn_scale"])
        if not case["grad"]:
            return list(ext.attn_sink_rope(s["q"], s["k"], s["positions"], s["inv_freq"], **kw))
        y = ext.attn_sink_rope_func(s["q"], s["k"], s["positions"], s["inv_freq"], **kw)
        g = torch.autograd.grad(y, (s["q"], s["k"]), (s["dq"], s["dk"]))
        return [y[0].detach(), y[1].detach(), *g]
    if op == "append":
        q = ext.attn_sink_rope_kv_append(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"],
                                         s["seqlens"], s["inv_freq"], cu_new=s["cu"], max_new=s["max_new"],
                                         interleaved=case["interleaved"], attn_scale=s["attn_scale"])
        return [q, s["k_cache"], s["v_cache"]]
    if op == "tree":
        return list(ext.attn_sink_tree_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["seqlens"],
                                             s["parents"], s["max_new"], s["max_len"], sink=s["sink"],
                                             win_first=case["first"], win_last=case["last"]))
    if op == "accept":
        ext.attn_sink_kv_compact(s["k_cache"], s["v_cache"], s["table"], s["src"], s["counts"], base=s["base"])
        return [s["k_cache"], s["v_cache"]]
    if op == "weights":
        out, lse = ext.attn_sink_decode_paged_weights(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seqlens"],
                                                      s["weights"], s["sink"], case["first"], case["last"])
        return [out, lse, s["weights"]]
    new, kept = ext.attn_sink_evict_paged(s["k_cache"], s["v_cache"], s["table"], s["seqlens"], s["weights"],
                                          case["budget"], keep_first=case["first"], keep_last=case["last"],
                                          weights_out=s["weights_out"])
    return [new, kept, s["weights_out"], s["k_cache"], s["v_cache"]]


def run(s):
    if own:
        return _own(s)
    return globals()["_plain_" + s["op"]](s)


# ---------------------------------------------------------------------------
# What a pass cannot do without.


def _visible(length, case):
    if case["last"] <= 0 or length <= case["first"] + case["last"]:
        return length
    return case["first"] + case["last"]


def work(case):
    op, d = case["op"], case["d"]
    if op == "rope":
        n = case["tokens"] * (case["hq"] + case["hkv"]) * (2 if case["grad"] else 1)
        return {"bytes": n * d * 2 * 2 + case["tokens"] * 4, "flops": n * case["rotary"] * 3}
    lens, hkv = lengths(case), case["hkv"]
    row = hkv * d * 2  # one token's keys
    if op == "append":
        rows = sum(n for _, n in lens)
        return {"bytes": rows * (case["hq"] * d * 2 * 2 + 4 * row), "flops": rows * (case["hq"] + hkv) * case["rotary"] * 3}
    if op == "tree":
        seen = sum(_visible(p + n, case) for p, n in lens)
        pairs = sum(n * _visible(p + n // 2, case) for p, n in lens)
        rows = sum(n for _, n in lens)
        return {"bytes": seen * 2 * row + rows * case["hq"] * (d * 4 + 4), "flops": 4 * d * case["hq"] * pairs}
    if op == "accept":
        mean = min(8, case["n_lo"]) / 2
        return {"bytes": case["batch"] * mean * 4 * row, "flops": 0}
    heads = hkv if case["per_head"] else 1
    if op == "weights":
        seen = sum(_visible(p, case) for p, _ in lens)
        return {"bytes": seen * (2 * row + 8 * heads) + case["batch"] * case["hq"] * d * 4, "flops": 4 * d * case["hq"] * seen}
    full = [p for p, _ in lens if p > case["budget"]]
    moved = len(full) * (case["budget"] - case["first"])
    cap = max(p for p, _ in lens)
    return {"bytes": moved * 4 * row + sum(p for p, _ in lens) * heads * 4
            + case["batch"] * heads * (case["budget"] + cap) * 4, "flops": 0}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, request by request.


def _exact_rotated(x, positions, inv_freq, scale, interleaved, sign=1.0):
    h = inv_freq.numel()
    turn = torch.polar(torch.full((positions.numel(), h), scale, dtype=torch.float64, device=x.device),
                       sign * torch.outer(positions.double(), inv_freq))[:, None, :]
    y = x.double().clone()
    if interleaved:
        z = torch.complex(y[..., 0:2 * h:2].contiguous(), y[..., 1:2 * h:2].contiguous()) * turn
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :h].contiguous(), y[..., h:2 * h].contiguous()) * turn
        y[..., :h], y[..., h:2 * h] = z.real, z.imag
    return y


def _tokens(cache, table, b, length):
    """The first `length` tokens of request b, (length, KV heads, d)."""
    page = cache.shape[1]
    return cache[table[b, :-(-length // page)].long()].reshape(-1, *cache.shape[2:])[:length]


def _exact_attention(q, k, v, seen, sink):
    """q (n, hq, d), k / v (t, hkv, d), seen (n, t); returns out (n, hq, d), log-sum-exp (hq, n), weights (hq, n, t)."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    k, v = (x.double().repeat_interleave(group, 1).transpose(0, 1) for x in (k, v))
    x = torch.matmul(q.double().transpose(0, 1), k.transpose(1, 2)) / math.sqrt(d)
    x = torch.where(seen, x, -math.inf)
    lse = torch.logsumexp(x, -1)
    if sink is not None:
        lse = torch.logaddexp(lse, sink.double()[:, None])
    p = torch.exp(x - lse[..., None])
    return torch.matmul(p, v).transpose(0, 1), lse, p


def _exact_seen(t, pos, case):
    if case["last"] <= 0:
        return t <= pos
    return (t <= pos) & ((t < case["first"]) | (t >= pos + 1 - case["last"]))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        a = (s["positions"], s["inv_freq"], s["attn_scale"], case["interleaved"])
        out = [_exact_rotated(s[n].detach(), *a) for n in ("q", "k")]
        return out + [_exact_rotated(s[n], *a, sign=-1.0) for n in ("dq", "dk")] if case["grad"] else out
    lens = lengths(case)
    if op == "append":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        q, row = [], 0
        for b, (p, n) in enumerate(lens):
            t = torch.arange(p, p + n, device="cuda")
            a = (t, s["inv_freq"], s["attn_scale"], case["interleaved"])
            q.append(_exact_rotated(s["q"][row:row + n], *a))
            page, at = s["table"][b].long()[t // case["page"]], t % case["page"]
            k[page, at] = _exact_rotated(s["k_new"][row:row + n], *a)
            v[page, at] = s["v_new"][row:row + n].double()
            row += n
        return [torch.cat(q), k, v]
    if op == "tree":
        out, lse, row = [], [], 0
        parents = s["parents"].tolist()
        for b, (p, n) in enumerate(lens):
            see, depth = torch.zeros(n, n, dtype=torch.bool), []
            for i in range(n):
                j = parents[row + i]
                if j >= 0:
                    see[i] = see[j]
                see[i, i] = True
                depth.append(0 if j < 0 else depth[j] + 1)
            pos = p + torch.tensor(depth, device="cuda")
            key = torch.cat([torch.arange(p, device="cuda"), pos])
            seen = torch.cat([torch.ones(n, p, dtype=torch.bool), see], 1).cuda() & _exact_seen(key, pos[:, None], case)
            some = seen.any(0)  # columns that no node sees are left out of the products
            k, v = (_tokens(s[c], s["table"], b, p + n)[some] for c in ("k_cache", "v_cache"))
            o, z, _ = _exact_attention(s["q"][row:row + n], k, v, seen[:, some], s["sink"])
            out.append(o)
            lse.append(z)
            row += n
        return [torch.cat(out), torch.cat(lse, 1)]
    if op == "weights":
        out, lse, w = [], [], s["weights"].double()
        for b, (p, _) in enumerate(lens):
            seen = _exact_seen(torch.arange(p, device="cuda"), p - 1, case)[None]
            k, v = (_tokens(s[c], s["table"], b, p) for c in ("k_cache", "v_cache"))
            o, z, prob = _exact_attention(s["q"][b:b + 1], k, v, seen, s["sink"])
            out.append(o)
            lse.append(z[:, 0])
            w[b, :, :p] += prob[:, 0].view(w.shape[1], -1, p).sum(1)
        return [torch.cat(out), torch.stack(lse), w]
    k, v = s["k_cache"].double(), s["v_cache"].double()
    page = case["page"]
    if op == "accept":
        for b in range(len(lens)):
            n = int(s["counts"][b])
            src = s["src"][b, :n].long()
            dst = int(s["base"][b]) + torch.arange(n, device="cuda")
            table = s["table"][b].long()
            for c in (k, v):
                c[table[dst // page], dst % page] = c[table[src // page], src % page]
        return [k, v]
    w = s["weights"].double()
    w_out = torch.zeros_like(w)
    kept = torch.full((*w.shape[:2], case["budget"]), -1, dtype=torch.int32, device="cuda")
    per = case["hkv"] // w.shape[1]
    for b, (p, _) in enumerate(lens):
        n, table = min(p, case["budget"]), s["table"][b].long()
        for h in range(w.shape[1]):
            keep = torch.zeros(p, dtype=torch.bool, device="cuda")
            keep[:case["first"]] = True
            keep[p - min(p, case["last"]):] = True
            free = n - int(keep.sum())
            rest = torch.nonzero(~keep).flatten()
            order = torch.argsort(-w[b, h, rest], stable=True)[:max(free, 0)]
            keep[rest[order]] = True
            src = torch.nonzero(keep).flatten()
            dst = torch.arange(n, device="cuda")
            kept[b, h, :n] = src.int()
            w_out[b, h, :n] = w[b, h, src]
            for c in (k, v):
                for j in range(h * per, (h + 1) * per):
                    c[table[dst // page], dst % page, j] = c[table[src // page], src % page, j]
    return [torch.tensor([min(p, case["budget"]) for p, _ in lens], dtype=torch.int32, device="cuda"), kept, w_out, k, v]
