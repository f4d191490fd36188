"""Inverse frequencies of rotary positions, scaled for long contexts.

Host arithmetic in 64 bits, done once when a model is set up; the rotation itself
is the library's ``attn_sink_rope``.
"""
import math

import torch

__all__ = ["attn_sink_rope_freqs"]


def attn_sink_rope_freqs(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_len=None, low=1.0, high=None,
                         attn_factor=None, device="cuda", round_ends=True):
    """(inv_freq, attn_scale): the rotary_dim / 2 inverse frequencies
    base^(-2i / rotary_dim) in radians per position as an fp64 tensor on ``device``,
    and the factor on the rotated part, changed by ``scaling`` to stretch a context
    of ``original_len`` positions by ``factor``:

    * None: unchanged.
    * "linear": every frequency divided by ``factor`` (positions squeezed).
    * "base": the base raised to base * factor^(r / (r - 2)), which leaves the first
      pair as it is and divides the last one's frequency by ``factor``.
    * "bands": by the turns n_i = original_len f_i / 2 pi that a pair makes in the
      original context: below ``low`` (1) divided by ``factor``, above ``high`` (4)
      kept, between them blended linearly in n_i.
    * "yarn": as "bands" but with the blend linear in the pair index i, between the
      indices of pairs with ``high`` (32) and ``low`` (1) turns (rounded outwards, or as
      they are where ``round_ends`` is false), and an attention factor of
      0.1 ln(factor) + 1.

    ``attn_factor`` replaces the attention factor (1, or that of "yarn")."""
    r = int(rotary_dim)
    if r < 2 or r % 2:
        raise ValueError(f"rotary_dim must be even and positive, got {rotary_dim}")
    if scaling not in (None, "linear", "base", "bands", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling == "base":
        if r == 2:
            raise ValueError('scaling "base" needs rotary_dim above 2')
        base = base * factor ** (r / (r - 2))
    freqs = [base ** (-2.0 * i / r) for i in range(r // 2)]
    scale = 1.0
    if scaling == "linear":
        freqs = [f / factor for f in freqs]
    elif scaling in ("bands", "yarn"):
        high = (4.0 if scaling == "bands" else 32.0) if high is None else high
        if original_len is None or original_len <= 0:
            raise ValueError(f'scaling "{scaling}" needs original_len')
        if not 0.0 < low < high:
            raise ValueError("0 < low < high is needed")
        if scaling == "bands":
            keep = [(original_len * f / (2 * math.pi) - low) / (high - low) for f in freqs]
        else:
            def index(turns):  # of the pair that makes so many turns
                return r * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
            first, last = index(high), index(low)
            if round_ends:
                first, last = math.floor(first), math.ceil(last)
            first, last = max(first, 0), min(last, r - 1)
            keep = [1.0 - (i - first) / max(last - first, 0.001) for i in range(r // 2)]
            scale = 0.1 * math.log(factor) + 1.0
        keep = [min(max(x, 0.0), 1.0) for x in keep]
        freqs = [f * x + f / factor * (1.0 - x) for f, x in zip(freqs, keep)]
    if attn_factor is not None:
        scale = float(attn_factor)
    return torch.tensor(freqs, dtype=torch.float64, device=device), scale
