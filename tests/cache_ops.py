"""Inputs shared by the tests of the operators around the paged cache."""
import torch


def paged(lens, hkv, d, page, seed=0, extra_pages=3, spare_columns=1):
    """Caches (CPU), a page table with pages in random order, and int32 lengths.
    Slots behind a request's last token and unused pages hold NaN."""
    g = torch.Generator().manual_seed(seed)
    n = [-(-t // page) for t in lens]
    pool = sum(n) + extra_pages
    perm = torch.randperm(pool, generator=g).int()
    table = torch.full((len(lens), max(n + [0]) + spare_columns), -1, dtype=torch.int32)
    k, v = (torch.full((pool, page, hkv, d), float("nan"), dtype=torch.bfloat16) for _ in range(2))
    at = 0
    for b, (t, m) in enumerate(zip(lens, n)):
        table[b, :m] = perm[at:at + m]
        at += m
        for c in (k, v):
            rows = torch.full((m * page, hkv, d), float("nan"), dtype=torch.bfloat16)
            rows[:t] = torch.randn(t, hkv, d, generator=g).bfloat16()
            c[table[b, :m].long()] = rows.view(m, page, hkv, d)
    return k, v, table, torch.tensor(lens, dtype=torch.int32)


def cu(lens):
    return torch.tensor([0] + list(torch.tensor(lens, dtype=torch.int64).cumsum(0)), dtype=torch.int32)


def same(a, b):
    """Bitwise equality of bf16 / fp32 tensors (NaN equal to itself)."""
    kind = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))
