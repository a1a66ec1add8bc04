"""Frequencies of rotary positions, plain and scaled for contexts longer than a model was trained on: the
angles that ``kv.make_rope`` takes.  Host arithmetic in float64."""
from __future__ import annotations

import math

import torch


def frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, trained: int = 0,
                fast: float = 32.0, slow: float = 1.0) -> torch.Tensor:
    """Radians a token of each of rot_dim / 2 pairs, base^(-2 i / rot_dim), scaled to a context of `factor` times the
    trained one:

    none    as they are
    linear  all divided by factor (positions interpolated)
    base    base times factor^(rot_dim / (rot_dim - 2)): the slowest pair's is divided by factor, the fastest kept
    ramp    pairs that turn at least `fast` times in the `trained` tokens are kept, those that turn at most `slow` times
            are divided by factor, and between them a blend that is linear in the pair's index; ``magnitude`` goes with it
    bands   the same with a blend that is linear in the number of turns
    """
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError(f"rot_dim={rot_dim} must be even and not negative")
    if not (base > 1.0 and factor >= 1.0):
        raise ValueError(f"base={base} must be above 1 and factor={factor} at least 1")
    if scaling not in ("none", "linear", "base", "ramp", "bands"):
        raise ValueError(f"scaling={scaling!r} is none of 'none', 'linear', 'base', 'ramp', 'bands'")
    if scaling in ("ramp", "bands") and not (trained > 0 and fast > slow > 0):
        raise ValueError("scaling by turns needs the trained length, and fast > slow > 0")
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    pair = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    f = base ** (-pair / max(1, rot_dim))
    if scaling == "linear":
        return f / factor
    if scaling in ("none", "base"):
        return f
    if scaling == "bands":
        keep = (f * trained / (2 * math.pi) - slow) / (fast - slow)
    else:
        def index(turns):  # of the pair that turns so many times in the trained tokens
            return rot_dim * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))
        # (the end may lie behind the last pair, which then keeps a part; the published method ends at rot_dim - 1)
        lo, hi = max(0.0, math.floor(index(fast))), min(rot_dim - 1.0, math.ceil(index(slow)))
        if hi <= 0.0:  # every pair turns at most `slow` times
            return f / factor
        keep = 1.0 - (pair / 2 - lo) / max(hi - lo, 1e-3)
    keep = keep.clamp(0.0, 1.0)
    return f * keep + f / factor * (1.0 - keep)


def magnitude(factor: float) -> float:
    """Factor of rotated queries and keys that goes with `ramp`: the scores of a longer context are sharpened by its
    square."""
    return 1.0 + 0.1 * math.log(max(1.0, factor))
