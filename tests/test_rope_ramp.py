"""Frequencies of scaling "ramp" against their definition, pair by pair, with the end of the blend among the pairs,
behind them and before them."""
import math

import pytest

from speculative_decode_verify_gdn_gb300 import rope

torch = pytest.importorskip("torch")


def kept(rot_dim, base, factor, trained, fast, slow):
    """Share of its frequency that each pair keeps: g = f (keep + (1 - keep) / factor)."""
    f = rope.frequencies(rot_dim, base)
    g = rope.frequencies(rot_dim, base, "ramp", factor, trained, fast, slow)
    return ((g / f - 1.0 / factor) / (1.0 - 1.0 / factor)).tolist()


def test_by_hand():
    """Frequencies 4^-i: in 442 tokens pair i turns 70.3 / 4^i times.  16 turns are those of pair 1.07, a quarter of a turn
    that of pair 4.07, behind the last pair 3: the blend goes from 1 to 5."""
    assert kept(8, 256.0, 4.0, 442, 16.0, 0.25) == pytest.approx([1.0, 1.0, 0.75, 0.5])
    # one turn: pair 3.07, so from 1 to 4; 20 turns: pair 0.91
    assert kept(8, 256.0, 4.0, 442, 16.0, 1.0) == pytest.approx([1.0, 1.0, 2 / 3, 1 / 3])
    assert kept(8, 256.0, 4.0, 442, 20.0, 4.0) == pytest.approx([1.0, 2 / 3, 1 / 3, 0.0])
    # no pair turns once in 6 tokens, and pair 0 alone does in 7
    assert kept(8, 256.0, 4.0, 6, 32.0, 1.0) == pytest.approx([0.0] * 4)
    assert kept(8, 256.0, 4.0, 7, 32.0, 1.0) == pytest.approx([1.0, 0.0, 0.0, 0.0])


@pytest.mark.parametrize("rot_dim", [2, 16, 64, 128])
@pytest.mark.parametrize("base", [500.0, 1e4, 1e6])
@pytest.mark.parametrize("trained", [3, 100, 4096, 65536, 262144, 1 << 24])
def test_every_pair(rot_dim, base, trained):
    """Pairs that turn `fast` times keep all, those that turn at most `slow` times nothing, and each step between them
    is the same.  1e-9: g / f has a few roundings of 2^-53, divided by 1 - 1 / factor."""
    keep = kept(rot_dim, base, 8.0, trained, 32.0, 1.0)
    turns = [trained / (2 * math.pi) * base ** (-2 * i / rot_dim) for i in range(rot_dim // 2)]
    for k, n in zip(keep, turns):
        assert -1e-9 <= k <= 1 + 1e-9
        if n >= 32.0 * (1 + 1e-12):
            assert k == pytest.approx(1.0, abs=1e-9)
        if n <= 1.0 - 1e-12:
            assert k == pytest.approx(0.0, abs=1e-9)
    # the blend's ends, from the turns that two neighbours' ratio gives
    pairs_per_e = rot_dim / (2 * math.log(base))
    lo = max(0, math.floor(pairs_per_e * math.log(trained / (2 * math.pi) / 32.0)))
    hi = min(rot_dim - 1, math.ceil(pairs_per_e * math.log(trained / (2 * math.pi))))
    for i, k in enumerate(keep):
        want = 0.0 if i >= hi else 1.0 if i <= lo else (hi - i) / (hi - lo)
        assert k == pytest.approx(want, abs=1e-9), i
