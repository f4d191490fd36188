"""What the operators of an 8-bit paged cache, of drafts and of pages are measured on.

Six operators: the write of new tokens into a cache held in 8 bits with a scale
for each block of tokens and KV head, single-token decode over such a cache,
attention of several new tokens a request over it, the verification of drafted
tokens against the target's probabilities, the step of a page table under
parallel samples (rows dropped back, forked, grown with copies of shared pages)
and the compaction of a pool's pages.  ``run`` computes them in elementary torch
operations, or with ``own`` through this package's entry points.
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
        # One decode step of 64 requests: the new tokens' keys and values written into the 8-bit cache.
        dict(name="append8_decode", op="append8", batch=64, len_lo=1, len_hi=4096, n_lo=1, n_hi=1, hkv=8, d=64, page=16,
             block=16, fmt="e4m3", lens=1),
        # Chunked prefill of 8 requests into an int8 cache with scales over half pages.
        dict(name="append8_extend", op="append8", batch=8, len_lo=0, len_hi=4096, n_lo=512, n_hi=8192, hkv=8, d=128,
             page=64, block=32, fmt="int8", lens=2),
        # A full serving batch's decode step over 1k to 32k tokens.
        dict(name="decode8_batch", op="decode8", batch=64, len_lo=1024, len_hi=32768, n_lo=1, n_hi=1, hq=64, hkv=8, d=64,
             page=16, block=16, fmt="e4m3", sink=True, first=0, last=0, lens=3),
        # Decode over long caches of which the first 1024 and the last 7168 tokens are seen.
        dict(name="decode8_window", op="decode8", batch=32, len_lo=8192, len_hi=65536, n_lo=1, n_hi=1, hq=32, hkv=8,
             d=128, page=64, block=64, fmt="int8", sink=False, first=1024, last=7168, lens=4),
        # One user's draft of 5 tokens in a row checked against a short conversation: latency.
        dict(name="extend8_one", op="extend8", batch=1, len_lo=2000, len_hi=2000, n_lo=5, n_hi=5, hq=64, hkv=8, d=64,
             page=16, block=16, fmt="e4m3", sink=True, first=0, last=0, lens=5),
        # Chunks of 4 requests' prompts behind what is cached of them.
        dict(name="extend8_chunks", op="extend8", batch=4, len_lo=0, len_hi=8192, n_lo=256, n_hi=1024, hq=64, hkv=8,
             d=64, page=16, block=16, fmt="e4m3", sink=True, first=0, last=0, lens=6),
        # One user's draft of 8 tokens in a row against a small vocabulary, drawn from a draft model: latency.
        dict(name="verify_one", op="verify", batch=1, n_lo=9, n_hi=9, vocab=32000, arity=1, sampled=True, dtype="fp32",
             lens=7),
        # A serving batch's drafted trees against a large vocabulary.
        dict(name="verify_trees", op="verify", batch=64, n_lo=8, n_hi=32, vocab=131072, arity=3, sampled=True,
             dtype="fp32", lens=8),
        # Four parallel samples of one request take a step: the losers' rows give way to the winners'.
        dict(name="beams_few", op="beams", batch=1, beams=4, len_lo=2000, len_hi=2000, grow=1, hkv=8, d=64, page=16,
             lens=9),
        # The same for 64 requests with 8 samples each, wide heads and large pages.
        dict(name="beams_batch", op="beams", batch=64, beams=8, len_lo=500, len_hi=4000, grow=4, hkv=8, d=128, page=64,
             lens=10),
        # A small pool, half of it free in between, brought together.
        dict(name="pool_few", op="pool", batch=8, len_lo=100, len_hi=2000, used=0.5, hkv=8, d=64, page=16, lens=11),
        # A large one.
        dict(name="pool_batch", op="pool", batch=64, len_lo=1024, len_hi=16384, used=0.7, hkv=8, d=64, page=16, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append8", "decode8", "extend8", "verify", "beams", "pool"))
    hq, hkv, d = rng.choice(HEADS)
    page = rng.choice((8, 16, 32, 64, 128))
    lens = rng.randrange(1 << 30)
    cache = dict(hkv=hkv, d=d, page=page, block=page // rng.choice((1, 1, 2, 4)), fmt=rng.choice(("e4m3", "int8")))
    window = rng.choice(((0, 0), (0, 0), (1024, 7168), (4, 509), (0, 1000)))
    attend = dict(hq=hq, sink=rng.random() < 0.5, first=window[0], last=window[1])
    if op == "append8":
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4000)
        return dict(op=op, batch=_log_int(rng, 1, 64 if new == 1 else 8), len_lo=0, len_hi=_log_int(rng, 16, 4096),
                    n_lo=max(1, new // 3), n_hi=new, lens=lens, **cache)
    if op == "decode8":
        hi = _log_int(rng, 64, 32000)
        return dict(op=op, batch=_log_int(rng, 1, 32), len_lo=max(1, hi // 8), len_hi=hi, n_lo=1, n_hi=1, lens=lens,
                    **cache, **attend)
    if op == "extend8":
        n = _log_int(rng, 2, 600)
        hi = _log_int(rng, 16, 6000)
        return dict(op=op, batch=_log_int(rng, 1, 4 if n > 64 else 16), len_lo=hi // 3, len_hi=hi, n_lo=(n + 1) // 2,
                    n_hi=n, lens=lens, **cache, **attend)
    if op == "verify":
        n = _log_int(rng, 2, 33)
        return dict(op=op, batch=_log_int(rng, 1, 32), n_lo=(n + 1) // 2, n_hi=n, vocab=_log_int(rng, 300, 120000),
                    arity=rng.choice((1, 1, 2, 4)), sampled=rng.random() < 0.6,
                    dtype=rng.choice(("fp32", "fp32", "bf16", "fp16")), lens=lens)
    if op == "beams":
        hi = _log_int(rng, 20, 4000)
        return dict(op=op, batch=_log_int(rng, 1, 32), beams=rng.choice((2, 3, 4, 8)), len_lo=hi // 3, len_hi=hi,
                    grow=rng.choice((1, 1, 2, 7, page)), hkv=hkv, d=d, page=page, lens=lens)
    hi = _log_int(rng, 50, 8000)
    return dict(op=op, batch=_log_int(rng, 1, 32), len_lo=hi // 4, len_hi=hi, used=rng.uniform(0.1, 0.95), hkv=hkv, d=d,
                page=page, lens=lens)


def lengths(case):
    """(cached tokens before the new ones, new tokens or drafted nodes) of every request, fixed by the case."""
    rng = random.Random(case["lens"])
    lo, hi = case.get("n_lo", 0), case.get("n_hi", 0)
    return [(rng.randint(case.get("len_lo", 0), case.get("len_hi", 0)), rng.randint(lo, hi)) for _ in range(case["batch"])]


# ---------------------------------------------------------------------------
# Inputs.

DTYPES = dict(fp32=torch.float32, bf16=torch.bfloat16, fp16=torch.float16)
CODES = dict(e4m3=torch.float8_e4m3fn, int8=torch.int8)
MIN_EXP = -64  # of a block's scale


class _Gen:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda", dtype=torch.bfloat16)

    def uniform(self, *shape, dtype=torch.float32):
        return torch.rand(*shape, generator=self.g, device="cuda", dtype=dtype)

    def below(self, n, *shape):
        return torch.randint(0, n, shape, generator=self.g, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _needed(top, fmt):
    """The smallest power of two, 2^MIN_EXP at least, at which `top` (fp32) has a code."""
    f, e = torch.frexp(top)
    e = e - 9 + (f > 0.875).int() if fmt == "e4m3" else e - 7 + (f > 127 / 128).int()  # 448 = 0.875 2^9
    e = torch.where(top > 0, e.clamp(min=MIN_EXP), MIN_EXP)
    return torch.ldexp(torch.ones_like(top), e)


def _coded(x, fmt):
    """Codes of fp32 values in units of their scale, to nearest, ties to even."""
    return x.to(torch.float8_e4m3fn) if fmt == "e4m3" else x.round().to(torch.int8)


def _bytes(codes):
    return codes.view(torch.int8)  # what is only moved is moved as bytes


def _values(data, fmt):
    return data.view(CODES[fmt]).float()


def _table(gen, page, total, pool=None):
    """A page table for requests of `total` tokens, pages in random order in a pool of just that size, or `pool`."""
    n = torch.tensor([-(-t // page) for t in total], device="cuda")
    held = int(n.sum())
    pool = max(held, pool or 1)
    perm = torch.randperm(pool, generator=gen.g, device="cuda").int()
    at = torch.arange(max(1, int(n.max())), device="cuda")[None, :].expand(len(total), -1)
    start = (n.cumsum(0) - n)[:, None]
    table = torch.where(at < n[:, None], perm[(start + at).clamp(max=pool - 1)], -1).int().contiguous()
    return table, pool


def _cache8(gen, case, pool):
    """One 8-bit cache of normal values, some blocks larger than others: codes and scales."""
    shape = (pool, case["page"] // case["block"], case["block"], case["hkv"], case["d"])
    x = gen.normal(*shape) * torch.exp2(gen.uniform(pool, shape[1], 1, case["hkv"], 1) * 4 - 2).bfloat16()
    scale = _needed(x.abs().amax((2, 4)).float(), case["fmt"])
    codes = _coded(x.float() / scale[:, :, None, :, None], case["fmt"])
    return codes.view(pool, case["page"], case["hkv"], case["d"]), scale


def _prepare_verify(case, gen, s):
    """Probabilities of a target and of a draft model that is near it, nodes hung on earlier ones, tokens drawn from the
    draft model (or, without one, from the likelier ones)."""
    lens = [n for _, n in lengths(case)]
    rows, vocab, dtype = sum(lens), case["vocab"], DTYPES[case["dtype"]]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0)
    s["cu"], s["max_nodes"] = cu.int(), max(lens)
    x = torch.randn(rows, vocab, generator=gen.g, device="cuda").mul_(3.0)
    s["target"] = x.softmax(-1).to(dtype)
    y = x.add_(torch.randn(rows, vocab, generator=gen.g, device="cuda").mul_(0.5)).softmax(-1)
    s["draft"] = y.to(dtype) if case["sampled"] else None
    row = torch.arange(rows, device="cuda")
    first = cu[torch.bucketize(row, cu[1:], right=True)]
    node = row - first
    # a node hangs on the one that many places before it, up to `arity` siblings
    parent = torch.div(node - 1, case["arity"], rounding_mode="floor")
    s["parents"] = parent.clamp(min=-1).int()
    cum = y[(first + parent).clamp(min=0)].cumsum_(-1)
    u = gen.uniform(rows, 1) * cum[:, -1:]
    s["tokens"] = (cum <= u).sum(-1).clamp(max=vocab - 1).int()
    s["u"], s["u_next"] = gen.uniform(rows), gen.uniform(case["batch"])
    s["base"] = gen.below(5000, case["batch"]).int()


def _prepare_beams(case, gen, s):
    """Every request's samples share its full pages and hold what follows in pages of their own."""
    page, beams, grow = case["page"], case["beams"], case["grow"]
    lens = [p for p, _ in lengths(case) for _ in range(beams)]
    full = torch.tensor([n // page for n in lens], device="cuda")  # shared pages of a row's request
    n = torch.tensor([-(-(x + grow) // page) for x in lens], device="cuda")
    rows = len(lens)
    group = torch.arange(rows, device="cuda") // beams
    lead = torch.arange(rows, device="cuda") % beams == 0
    mine = torch.where(lead, n, n - full)
    most = int((n - full).sum() + full.sum() // beams)
    pool = most + rows * (1 + grow // page) + 8
    perm = torch.randperm(pool, generator=gen.g, device="cuda").int()
    start = mine.cumsum(0) - mine
    at = torch.arange(int(n.max()), device="cuda")[None, :]
    head = (start - torch.where(lead, 0, full))[:, None] + at
    index = torch.where(at < full[:, None], start[group * beams][:, None] + at, head)
    s["table"] = torch.where(at < n[:, None], perm[index.clamp(0, pool - 1)], -1).int().contiguous()
    s["refs"] = torch.zeros(pool + 1, dtype=torch.int32, device="cuda").index_add_(
        0, torch.where(s["table"] < 0, pool, s["table"]).view(-1).long(),
        torch.ones(s["table"].numel(), dtype=torch.int32, device="cuda"))[:pool].contiguous()
    s["lens"] = _i32(lens)
    s["grown"] = s["lens"] + grow
    s["src"] = (group * beams + gen.below(beams, rows)).int()
    s["k_cache"], s["v_cache"] = (gen.normal(pool, page, case["hkv"], case["d"]) for _ in range(2))


def prepare(case, seed):
    gen, op = _Gen(seed), case["op"]
    s = dict(case=case, op=op)
    if op == "verify":
        _prepare_verify(case, gen, s)
        return s
    if op == "beams":
        _prepare_beams(case, gen, s)
        return s
    lens = lengths(case)
    total = [p + n for p, n in lens]
    if op == "pool":
        held = sum(-(-t // case["page"]) for t in total)
        s["table"], pool = _table(gen, case["page"], total, int(held / case["used"]))
        s["refs"] = torch.zeros(pool, dtype=torch.int32, device="cuda")
        s["refs"][s["table"][s["table"] >= 0].long()] = 1
        s["lens"] = _i32(total)
        s["k_cache"], s["v_cache"] = (gen.normal(pool, case["page"], case["hkv"], case["d"]) for _ in range(2))
        return s
    s["table"], pool = _table(gen, case["page"], total)
    (s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]) = (_cache8(gen, case, pool) for _ in range(2))
    s["seqlens"] = _i32(total)
    s["max_len"], s["max_new"] = max(total), max(n for _, n in lens)
    new = torch.tensor([n for _, n in lens], device="cuda")
    s["cu"] = torch.cat([new.new_zeros(1), new.cumsum(0)]).int()
    rows = sum(n for _, n in lens)
    if op == "append8":
        s["k_new"], s["v_new"] = (gen.normal(rows, case["hkv"], case["d"]) * torch.exp2(gen.uniform(rows, 1, 1) * 4 - 2).bfloat16()
                                  for _ in range(2))
        return s
    s["q"] = gen.normal(rows, case["hq"], case["d"])
    s["sink"] = gen.uniform(case["hq"]) * 6 - 2 if case["sink"] else None
    return s


# ---------------------------------------------------------------------------
# The plain forms: 32 bits; probabilities' sums and comparisons in 64.


def _slot(s, b, t):
    page = s["case"]["page"]
    return s["table"][b, t // page].long() * page + t % page


def _new_rows(s):
    """Request, token and position in the request's new ones of every new row."""
    cu = s["cu"].long()
    row = torch.arange(int(s["k_new" if "k_new" in s else "q"].shape[0]), device="cuda")
    b = torch.bucketize(row, cu[1:], right=True)
    return b, s["seqlens"].long()[b] - (cu[b + 1] - row), row - cu[b]


def _plain_append8(s):
    case = s["case"]
    fmt, block = case["fmt"], case["block"]
    b, t, _ = _new_rows(s)
    slot = _slot(s, b, t)
    # tokens that a request's first block already has
    prefix = (s["seqlens"] - (s["cu"][1:] - s["cu"][:-1])).long()[:, None]
    old_t = torch.div(prefix, block, rounding_mode="floor") * block + torch.arange(block, device="cuda")
    old = (old_t < prefix) & (s["seqlens"][:, None] > prefix)
    old_slot = _slot(s, torch.arange(prefix.shape[0], device="cuda")[:, None], torch.where(old, old_t, 0))
    for x in ("k", "v"):
        scale = s[x + "_scale"].view(-1, case["hkv"])
        data = _bytes(s[x + "_cache"]).view(-1, case["hkv"], case["d"])
        new = s[x + "_new"].float()
        held = data[old_slot], scale[old_slot // block]
        start = torch.div(t, block, rounding_mode="floor") * block
        scale[slot[start >= prefix[b, 0]] // block] = 0.0  # blocks without older tokens
        scale.scatter_reduce_(0, (slot // block)[:, None].expand(-1, case["hkv"]), _needed(new.abs().amax(-1), fmt), "amax")
        again = _coded(_values(held[0], fmt) * (held[1] / scale[old_slot // block])[..., None], fmt)
        data[old_slot[old]] = _bytes(again)[old]
        data[slot] = _bytes(_coded(new / scale[slot // block][..., None], fmt))
    return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _gathered(s, x):
    """Every request's cached tokens' values, padded: (batch, tokens, KV heads, d) in 32 bits."""
    case = s["case"]
    b = torch.arange(s["seqlens"].numel(), device="cuda")[:, None]
    t = torch.arange(s["max_len"], device="cuda")[None, :]
    slot = _slot(s, b, torch.minimum(t, s["seqlens"].long()[:, None] - 1))
    codes = _bytes(s[x + "_cache"]).view(-1, case["hkv"], case["d"])[slot]
    return _values(codes, case["fmt"]) * s[x + "_scale"].view(-1, case["hkv"])[slot // case["block"]][..., None]


def _in_window(t, pos, case):
    seen = t <= pos
    if case["last"] > 0:
        seen = seen & ((t < case["first"]) | (t > pos - case["last"]))
    return seen


def _attend8(s):
    """Outputs (rows, query heads, d) and log-sum-exp (rows, query heads) of the last rows of every request."""
    case, n = s["case"], s["max_new"]
    batch, hq, hkv, d = s["seqlens"].numel(), case["hq"], case["hkv"], case["d"]
    b, pos_row, node = _new_rows(s)
    q = torch.zeros(batch, n, hq, d, device="cuda")
    q[b, node] = s["q"].float()
    q = q.view(batch, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    scores = (q @ _gathered(s, "k").permute(0, 2, 3, 1)).mul_(d ** -0.5).view(batch, hq, n, -1)
    pos = torch.zeros(batch, n, dtype=torch.long, device="cuda")
    pos[b, node] = pos_row
    seen = _in_window(torch.arange(s["max_len"], device="cuda"), pos[..., None], case)
    scores.masked_fill_(~seen[:, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    sink = None if s["sink"] is None else s["sink"][:, None, None]
    if sink is not None:
        top = torch.maximum(top, sink)
    e = scores.sub_(top).exp_()
    z = e.sum(-1, keepdim=True)
    if sink is not None:
        z = z + (sink - top).exp()
    out = e.div_(z).view(batch, hkv, -1, s["max_len"]) @ _gathered(s, "v").transpose(1, 2)
    out = out.view(batch, hq, n, d)[b, :, node].bfloat16()
    return out, (top + z.log()).view(batch, hq, n)[b, :, node]


def _plain_decode8(s):
    return list(_attend8(s))


def _plain_extend8(s):
    out, lse = _attend8(s)
    return [out, lse.t().contiguous()]


def _plain_verify(s):
    case, cu = s["case"], s["cu"].long()
    batch, n, rows, arity = case["batch"], s["max_nodes"], s["tokens"].numel(), case["arity"]
    row = torch.arange(rows, device="cuda")
    b = torch.bucketize(row, cu[1:], right=True)
    node = row - cu[b]
    up = (cu[b] + s["parents"].long()).clamp(min=0)  # the parent's row; the first node's is of no account
    up = torch.where(node == 0, row, up)
    x = s["tokens"].long()
    kin = (up[:, None] == up[None, :]) & (row[:, None] > row[None, :]) & (node[None, :] > 0) & (node[:, None] > 0)
    rank = kin.sum(1)  # earlier siblings
    kids = torch.zeros(rows, dtype=torch.long, device="cuda").index_add_(0, up, (node > 0).long())
    p, u = s["target"].double().clamp(0, 1), s["u"].double()
    px = p[up, x]
    if s["draft"] is None:  # a sibling's token is taken out of the target's row when it is refused
        again = (kin & (x[:, None] == x[None, :])).any(1)
        gone = torch.where(again, 0.0, px)
        z = 1.0 - (kin * gone).sum(1)
        fits = (u * z < px) & ~again
        left = p.clone()
        left[up[node > 0], x[node > 0]] = 0.0
    else:  # what the draft's rows cover is taken out, once for every refused sibling
        q = s["draft"].double().clamp(0, 1)
        cover, mass = torch.zeros_like(u), torch.ones_like(u)
        fits = torch.zeros_like(rank, dtype=torch.bool)
        left = p.clone()
        for k in range(arity):
            now = u * q[up, x] * mass[up] < (px - cover[up] * q[up, x]).clamp(min=0)
            fits = torch.where(rank == k, now, fits)
            more = kids > k
            cover = torch.where(more, cover + mass, cover)
            left = torch.where(more[:, None], (p - cover[:, None] * q).clamp_(min=0), left)
            mass = torch.where(more, left.sum(-1), mass)
    took = fits & ~(kin & fits[None, :]).any(1)
    good, ptr = torch.where(node == 0, True, took), up.clone()
    for _ in range(8):  # every ancestor taken: their chain is halved each time
        good, ptr = good & good[ptr], ptr[ptr]
    grid = torch.full((batch, n), n, device="cuda")
    grid[b, node] = torch.where(good, node, n)
    path = grid.sort(1).values
    count = (path < n).sum(1)
    last = cu[:-1] + torch.where(path < n, path, -1).amax(1)
    src = torch.where(path < n, s["base"].long()[:, None] + path, -1)
    w = left[last]
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p[last])
    cum = w.cumsum(1)
    token = (cum <= s["u_next"].double()[:, None] * cum[:, -1:]).sum(1).clamp(max=case["vocab"] - 1)
    return [src.int(), count.int(), token.int()]


def _pages(case, tokens):
    return torch.div(tokens.long() + case["page"] - 1, case["page"], rounding_mode="floor")


def _count(refs, table, live, sign):
    """Adds `sign` to the reference counts of the table's live entries."""
    pages = torch.where(live, table, refs.numel()).view(-1).long()
    more = torch.zeros(refs.numel() + 1, dtype=torch.int32, device="cuda")
    refs += sign * more.index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))[:-1]


def _plain_beams(s):
    case, table, refs = s["case"], s["table"], s["refs"]
    rows, width = table.shape
    at = torch.arange(width, device="cuda")[None, :]
    held, want = _pages(case, s["lens"])[:, None], _pages(case, s["grown"])[:, None]
    # the last tokens are dropped
    drop = (at >= held) & (at < want)
    _count(refs, table, drop, -1)
    table = torch.where(drop, -1, table)
    # row b goes on from row src[b]
    _count(refs, table, at < held, -1)
    table = table[s["src"].long()].clone()
    _count(refs, table, at < held, 1)
    # pages for the next tokens: a shared page that is partly filled is copied first, but for its last holder
    part = (s["lens"] % case["page"] != 0) & (s["grown"] > s["lens"])
    row = torch.arange(rows, device="cuda")
    mine = table[row, (held[:, 0] - 1).clamp(min=0)].long()
    key = torch.where(part, mine, refs.numel())
    users = torch.zeros(refs.numel() + 1, dtype=torch.int32, device="cuda").index_add_(0, key, torch.ones_like(key).int())
    keeper = torch.full_like(users, -1).scatter_reduce_(0, key, row.int(), "amax")
    copy = part & ~((users[key] == torch.nn.functional.pad(refs, (0, 1))[key]) & (keeper[key] == row))
    need = copy.long() + (want - held)[:, 0]
    short = (need.sum() - (refs == 0).sum()).clamp(min=0)
    first = need.cumsum(0) - need
    free = (refs == 0).int().sort(descending=True, stable=True).indices
    new = (at >= held) & (at < want) | copy[:, None] & (at == held - 1)
    rank = first[:, None] + new.long().cumsum(1) - 1
    table = torch.where(new, free[rank.clamp(0, free.numel() - 1)].int(), table)
    refs -= torch.zeros_like(users).index_add_(0, torch.where(copy, mine, refs.numel()), torch.ones_like(mine).int())[:-1]
    _count(refs, table, new, 1)
    to = table[row, (held[:, 0] - 1).clamp(min=0)].long()[copy]
    for name in ("k_cache", "v_cache"):
        s[name][to] = s[name][mine[copy]]
    s["table"] = table
    return [table, refs, s["lens"][s["src"].long()], short.view(1).int(), s["k_cache"], s["v_cache"]]


def _plain_pool(s):
    table, refs = s["table"].clone(), s["refs"].clone()
    used = refs > 0
    held = used.sum()
    page = torch.arange(refs.numel(), device="cuda")
    from_ = page[used & (page >= held)]
    to = page[~used & (page < held)]
    new = page.clone()
    new[from_] = to
    table = torch.where(table >= 0, new[table.clamp(min=0).long()].int(), table)
    refs[to] = refs[from_]
    refs[from_] = 0
    for name in ("k_cache", "v_cache"):
        s[name][to] = s[name][from_]
    return [table, refs, held.view(1).int(), s["k_cache"], s["v_cache"]]


# ---------------------------------------------------------------------------
# One pass.


def _own(s):
    import paged_kv_sink_gb300 as ext
    case, op = s["case"], s["op"]
    if op == "verify":
        return list(ext.attn_sink_verify_draft(s["target"], s["tokens"], s["parents"], s["cu"], s["u"], s["u_next"],
                                               s["max_nodes"], draft=s["draft"], base=s["base"]))
    if op == "beams":
        caches, page = (s["k_cache"], s["v_cache"]), case["page"]
        ext.attn_sink_pages_release(s["table"], s["refs"], s["grown"], s["lens"], page)
        table, lens = ext.attn_sink_pages_fork(s["table"], s["refs"], s["lens"], s["src"], page)
        missing = ext.attn_sink_pages_reserve(caches, table, s["refs"], lens, s["grown"], page)
        s["table"] = table
        return [table, s["refs"], lens, missing, *caches]
    if op == "pool":
        caches, table, refs = (s["k_cache"], s["v_cache"]), s["table"].clone(), s["refs"].clone()
        held = ext.attn_sink_pages_compact(caches, table, refs, s["lens"], case["page"])
        return [table, refs, held, *caches]
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    if op == "append8":
        ext.attn_sink_kv_append_q8(s["k_new"], s["v_new"], *cache, s["table"], s["seqlens"], cu_new=s["cu"],
                                   max_new=s["max_new"])
        return list(cache)
    if op == "decode8":
        return list(ext.attn_sink_decode_paged_q8(s["q"], *cache, s["table"], s["seqlens"], s["sink"], case["first"],
                                                  case["last"]))
    return list(ext.attn_sink_fwd_paged_q8(s["q"], *cache, s["table"], s["cu"], s["seqlens"], s["max_new"], s["max_len"],
                                           s["sink"], win_first=case["first"], win_last=case["last"]))


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
    op, lens = case["op"], lengths(case)
    if op == "verify":
        size = 4 if case["dtype"] == "fp32" else 2
        each = (2 if case["sampled"] else 1) * size
        rows = sum(n for _, n in lens)
        return {"bytes": case["batch"] * (case["vocab"] * each + 12) + rows * (2 * each + 16), "flops": case["batch"] * case["vocab"] * 4}
    d, hkv = case["d"], case["hkv"]
    if op in ("beams", "pool"):
        held = sum(-(-p // case["page"]) for p, _ in lens)
        size = 2 * case["page"] * hkv * d * 2  # K and V of a page
        if op == "pool":
            pool = int(held / case["used"])
            return {"bytes": 2 * size * held * (pool - held) / pool + 4 * (held + pool), "flops": 0}
        b = case["beams"]  # of b rows with random sources, those that find theirs taken copy its last page
        twins = b - b * (1 - (1 - 1 / b) ** b)
        part = sum(1 for p, _ in lens if p % case["page"])
        return {"bytes": 2 * size * part * twins + 4 * held * b * 2, "flops": 0}
    row = 2 * hkv * (d + 4 / case["block"])  # a token's keys and values with their share of the scales
    rows = sum(n for _, n in lens)
    if op == "append8":
        return {"bytes": rows * (4 * hkv * d + row), "flops": rows * hkv * d * 4}
    seen = sum(_visible(p + n, case) for p, n in lens)
    pairs = sum(n * _visible(p + n // 2, case) for p, n in lens)
    return {"bytes": seen * row + rows * case["hq"] * (d * 4 + 4), "flops": 4 * d * case["hq"] * pairs}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, request by request.


def _exact_code(x, scale, fmt):
    """What the nearest code stands for in units of the scale, ties to even, in 64 bits."""
    y = x / scale
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step).mul(step).clamp(-448, 448)


def _exact_scale(top, fmt):
    most = 448.0 if fmt == "e4m3" else 127.0
    e = MIN_EXP
    while most * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def _exact_append8(case, s):
    fmt, block, page = case["fmt"], case["block"], case["page"]
    table, out = s["table"].tolist(), []
    for x in ("k", "v"):
        scale = s[x + "_scale"].double()
        data = _values(_bytes(s[x + "_cache"]), fmt).double()
        new, row = s[x + "_new"].double(), 0
        for b, (p, n) in enumerate(lengths(case)):
            for t0 in range(p // block * block, p + n, block):
                pg, at = table[b][t0 // page], t0 % page
                lo, hi = max(p, t0), min(p + n, t0 + block)
                rows = new[row + lo - p:row + hi - p]
                top = rows.abs().amax((0, 2))
                need = torch.tensor([_exact_scale(v, fmt) for v in top.tolist()], dtype=torch.float64, device="cuda")
                here = at // block
                if lo > t0:
                    need = torch.maximum(need, scale[pg, here])
                    old = data[pg, at:at + lo - t0] * scale[pg, here][:, None]
                    data[pg, at:at + lo - t0] = _exact_code(old, need[:, None], fmt)
                scale[pg, here] = need
                data[pg, at + lo - t0:at + hi - t0] = _exact_code(rows, need[:, None], fmt)
            row += n
        out.append((data.to(torch.int8) if fmt == "int8" else data, scale))
    (k, ks), (v, vs) = out
    return [k, v, ks, vs]


def _exact_attend8(case, s):
    out, lse, row = [], [], 0
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    for b, (p, n) in enumerate(lengths(case)):
        pages = s["table"][b, :-(-(p + n) // page)].long()
        k, v = ((_values(_bytes(s[x + "_cache"])[pages], case["fmt"]).double()
                 * s[x + "_scale"][pages].double().repeat_interleave(case["block"], 1)[..., None])
                .reshape(-1, hkv, d)[:p + n].transpose(0, 1) for x in ("k", "v"))
        pos = torch.arange(p, p + n, device="cuda")
        t = torch.arange(p + n, device="cuda")
        seen = t <= pos[:, None]
        if case["last"] > 0:
            seen &= (t < case["first"]) | (t >= pos[:, None] + 1 - case["last"])
        o, z = [], []
        for h in range(hq):
            a = (s["q"][row:row + n, h].double() @ k[h * hkv // hq].t() / math.sqrt(d)).masked_fill(~seen, -math.inf)
            c = torch.logsumexp(a, -1)
            if s["sink"] is not None:
                c = torch.logaddexp(c, s["sink"][h].double())
            o.append(torch.exp(a - c[:, None]) @ v[h * hkv // hq])
            z.append(c)
        out.append(torch.stack(o, 1))
        lse.append(torch.stack(z, 1))
        row += n
    return torch.cat(out), torch.cat(lse)


def _exact_verify(case, s):
    cu, parents, tokens = s["cu"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    u, base = s["u"].tolist(), s["base"].tolist()
    src = torch.full((case["batch"], s["max_nodes"]), -1, dtype=torch.int32)
    counts, following = [], []
    for b in range(case["batch"]):
        r0, n = cu[b], cu[b + 1] - cu[b]
        path, w = [0], None
        while True:
            i = path[-1]
            p = s["target"][r0 + i].double()
            w, mass, cover, took = p, 1.0, 0.0, None
            q = None if s["draft"] is None else s["draft"][r0 + i].double()
            for c in range(i + 1, n):
                if parents[r0 + c] != i:
                    continue
                x = tokens[r0 + c]
                if float(w[x]) > u[r0 + c] * mass * (1.0 if q is None else float(q[x])):
                    took = c
                    break
                if q is None:
                    mass -= float(w[x])
                    w = w.clone()
                    w[x] = 0.0
                else:
                    cover += mass
                    w = torch.clamp(p - cover * q, min=0.0)
                    mass = float(w.sum())
            if took is None:
                break
            path.append(took)
        cum = torch.cumsum(w, 0)
        counts.append(len(path))
        src[b, :len(path)] = torch.tensor(path, dtype=torch.int32) + base[b]
        following.append(int(torch.searchsorted(cum, cum[-1:] * float(s["u_next"][b]), right=True)))
    i32 = dict(dtype=torch.int32, device="cuda")
    return [src.cuda(), torch.tensor(counts, **i32), torch.tensor(following, **i32)]


def _exact_beams(case, s):
    page, grow = case["page"], case["grow"]
    table, refs, lens, src = (s[x].tolist() for x in ("table", "refs", "lens", "src"))
    k, v = s["k_cache"].clone(), s["v_cache"].clone()
    for row, n in zip(table, lens):
        for i in range(-(-n // page), -(-(n + grow) // page)):
            refs[row[i]] -= 1
            row[i] = -1
        for i in range(-(-n // page)):
            refs[row[i]] -= 1
    table = [list(table[b]) for b in src]
    for row in table:
        for pg in row:
            if pg >= 0:
                refs[pg] += 1
    free = iter([i for i, r in enumerate(refs) if r == 0])
    for row, n in zip(table, lens):
        last = n // page
        if n % page and refs[row[last]] > 1:
            refs[row[last]] -= 1
            to = next(free)
            k[to], v[to] = s["k_cache"][row[last]], s["v_cache"][row[last]]
            row[last], refs[to] = to, 1
        for i in range(-(-n // page), -(-(n + grow) // page)):
            row[i] = next(free)
            refs[row[i]] = 1
    return [_i32(table), _i32(refs), _i32([lens[b] for b in src]), _i32([0]), k, v]


def _exact_pool(case, s):
    table, refs = s["table"].tolist(), s["refs"].tolist()
    k, v = s["k_cache"].clone(), s["v_cache"].clone()
    held = sum(r > 0 for r in refs)
    to = [i for i in range(held) if refs[i] == 0]
    from_ = [i for i in range(held, len(refs)) if refs[i] > 0]
    move = dict(zip(from_, to))
    k[to], v[to] = s["k_cache"][from_], s["v_cache"][from_]
    for a, b in move.items():
        refs[b], refs[a] = refs[a], 0
    return [_i32([[move.get(p, p) for p in row] for row in table]), _i32(refs), _i32([held]), k, v]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("decode8", "extend8"):
        out, lse = _exact_attend8(case, s)
        return [out, lse if op == "decode8" else lse.t().contiguous()]
    return globals()["_exact_" + op](case, s)
