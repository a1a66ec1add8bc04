"""Host side of norms and rotation, reserve, append and prefill attention, and pins of their oracle.

Every library call here is built to fail validation, which happens before the library touches CUDA, or runs
on the host alone: no GPU is needed and no kernel is launched."""
import ctypes
import fractions
import math

import numpy as np
import pytest

from oracle import prompt_oracle as O
from speculative_decode_verify_gdn_gb300 import build, gdn, kv, rope
from speculative_decode_verify_gdn_gb300.kv_runtime import PagedCache

torch = pytest.importorskip("torch")
INV, UNS, ALIAS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_ALIAS
BASE = dict(B=2, K=4, Hq=4, Hkv=2, D=64, page_size=16, n_pages=10, max_pages=4, n_slots=3, n_layers=2)
P, MB = 1 << 32, 1 << 24     # never dereferenced
BIG = ctypes.c_uint64(1 << 40)
N = 8                        # B * K, and the packed tokens


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return kv.load_library()


def ptrs(n):
    return [P + i * MB for i in range(n)]


def dims(**over):
    return kv.make_kv_dims(**dict(BASE, **over))


def with_field(name, value, **over):
    d = dims(**over)
    setattr(d, name, value)
    return d


def turning(**over):
    r = dict(rot_dim=32, interleaved=0, magnitude=1.0, eps=1e-6, weight_offset=0.0, reserved=0, q_token_stride=256,
             q_head_stride=64, kv_token_stride=128, kv_head_stride=64)
    r.update(over)
    return kv.GdnRope(*(r[n] for n, _ in kv.GdnRope._fields_))


def ref(x):
    return None if x is None else ctypes.byref(x)


# arguments: turns q_weight k_weight q k v seq_len prefix_of win_len parent positions | q_out k_win v_win
def window(lib, d, a=None, r=None):
    return lib.gdn_attn_rope(ref(d), ref(turning() if r is None else r), *(ptrs(14) if a is None else a), None)


def reserve(lib, d, a=None, ws=BIG):
    return lib.gdn_kv_reserve(ref(d), *(ptrs(8) if a is None else a), ws, None)


# turns q_weight k_weight | cu q k v positions k_cache v_cache table seq_len prefix_of q_out
def append(lib, d, a=None, r=None, layer=0, n=N):
    a = ptrs(14) if a is None else a
    return lib.gdn_kv_append(ref(d), layer, ref(turning() if r is None else r), *a[:3], n, *a[3:], None)


# cu q k_cache v_cache table seq_len prefix_of | out lse workspace
def prefill(lib, d, a=None, layer=0, n=N, scale=0.125, ws=BIG, causal=1):
    a = ptrs(10) if a is None else a
    return lib.gdn_attn_prefill(ref(d), layer, n, *a[:7], causal, scale, *a[7:], ws, None)


CALLS = [window, reserve, append, prefill]


@pytest.mark.parametrize("name,value,status", [
    ("Hkv", 0, INV), ("D", 96, UNS), ("page_size", 24, UNS), ("n_pages", 0, INV), ("n_slots", 0, INV),
    ("max_pages", 0, INV), ("n_layers", 0, INV), ("dtype", 2, INV), ("B", -1, INV), ("B", 65536, INV), ("slot0", -1, INV),
    ("slot0", 2, INV), ("cache_token_stride", 60, INV), ("cache_head_stride", 8, INV)])
def test_dims_are_checked_by_every_call(lib, name, value, status):
    for call in CALLS:
        assert call(lib, with_field(name, value)) == status, call
        assert gdn.last_error() != ""


@pytest.mark.parametrize("call,name,value,status", [
    (window, "K", 0, UNS), (window, "K", 17, UNS), (window, "Hq", 0, INV), (window, "Hq", 5, UNS),
    (window, "q_token_stride", 200, INV), (window, "win_token_stride", 64, INV), (window, "win_token_stride", 130, INV),
    (append, "Hq", 5, UNS), (append, "q_token_stride", 248, INV), (prefill, "Hq", 0, INV), (prefill, "Hq", 258, UNS),
    (prefill, "q_token_stride", 258, INV)])
def test_dims_of_single_calls(lib, call, name, value, status):
    assert call(lib, with_field(name, value)) == status
    assert gdn.last_error() != ""


@pytest.mark.parametrize("name,value,status", [
    ("rot_dim", -8, INV), ("rot_dim", 72, INV), ("rot_dim", 20, UNS), ("rot_dim", 40, UNS), ("interleaved", 2, INV), ("reserved", 1, INV),
    ("magnitude", float("nan"), INV), ("magnitude", float("inf"), INV), ("eps", -1e-6, INV), ("eps", float("nan"), INV),
    ("weight_offset", float("inf"), INV), ("q_token_stride", 100, INV), ("q_head_stride", -64, INV),
    ("kv_token_stride", 12, INV), ("kv_head_stride", 1 << 36, INV)])
def test_rotations_are_checked(lib, name, value, status):
    for call in (window, append):
        assert call(lib, dims(), r=turning(**{name: value})) == status, call
        assert gdn.last_error() != ""


def check_pointers(lib, call, n, optional, align):
    for i in range(n):
        if i not in optional:
            a = ptrs(n)
            a[i] = None
            assert call(lib, dims(), a) == INV, i
            assert "NULL" in gdn.last_error() or "without" in gdn.last_error(), i
        a = ptrs(n)
        a[i] += align.get(i, 4) // 2
        assert call(lib, dims(), a) == INV and "aligned" in gdn.last_error(), i
    assert call(lib, None) == INV and "dims" in gdn.last_error()


def test_window_arguments(lib):
    rows = {i: 16 for i in (1, 2, 3, 4, 5, 11, 12, 13)}
    check_pointers(lib, window, 14, (1, 2, 6, 7, 8, 9, 10), {**rows, 0: 8})
    assert lib.gdn_attn_rope(ref(dims()), None, *ptrs(14), None) == INV
    for out in (11, 12, 13):
        for i in range(11):
            if i != out - 8:                       # (its own input: in place)
                a = ptrs(14)
                a[out] = a[i]
                assert window(lib, dims(), a) == ALIAS, (out, i)
        a = ptrs(14)
        a[out] = a[out - 8] + 16                   # shifted is not in place
        assert window(lib, dims(), a) == ALIAS, out
    a = ptrs(14)
    a[6] = a[10] = None                            # neither lengths nor positions
    assert window(lib, dims(), a) == INV and "seq_len" in gdn.last_error()
    for i, o in ((3, 11), (4, 12), (5, 13)):
        a = ptrs(14)
        a[o] = None
        assert window(lib, dims(), a) == INV and "output" in gdn.last_error()
        a = ptrs(14)
        a[i] = None
        assert window(lib, dims(), a) == INV and "input" in gdn.last_error()
    a = ptrs(14)
    for i in (3, 4, 5, 11, 12, 13):
        a[i] = None
    assert window(lib, dims(), a) == gdn.GDN_OK    # nothing to do
    assert window(lib, dims(B=0)) == gdn.GDN_OK


def test_rows_of_one_buffer_beside_one_another(lib):
    """Parts of a projection's rows rewritten in place: the parts may not touch.  The last buffer is made to
    overlap positions, so that an accepted placement still ends in a refusal."""
    step = 4 * 64 + 2 * 2 * 64

    def says(q=0, k=256, v=384, q_out=0, k_win=256, v_win=384, out_step=step, in_step=step):
        d = dims()
        d.q_token_stride = d.win_token_stride = out_step
        a = ptrs(14)
        for i, off in zip((3, 4, 5, 11, 12, 13), (q, k, v, q_out, k_win, v_win)):
            a[i] = P + 1024 * MB + 2 * off
        a[10] = a[13]                              # positions over v_win, looked at last
        assert window(lib, d, a, turning(q_token_stride=in_step, kv_token_stride=in_step)) == ALIAS
        return gdn.last_error()

    assert "positions" in says()
    assert "positions" not in says(q_out=8)        # not in place, and over q
    assert "positions" not in says(k_win=248)      # over the end of q
    assert "positions" not in says(out_step=step + 64)
    far = 1 << 20
    assert "positions" in says(q_out=far, k_win=far + 256, v_win=far + 384)
    assert "positions" not in says(q_out=far, k_win=far + 192, v_win=far + 384)


def test_append_arguments(lib):
    rows = {i: 16 for i in (1, 2, 4, 5, 6, 8, 9, 13)}
    check_pointers(lib, append, 14, (1, 2, 7, 12), {**rows, 0: 8})
    for layer in (-1, 2):
        assert append(lib, dims(), layer=layer) == INV and "layer" in gdn.last_error()
    for n in (-1, 1 << 31):
        assert append(lib, dims(), n=n) == INV and "n_tokens" in gdn.last_error()
    for out in (8, 9, 13):
        for i in (0, 1, 2, 3, 4, 5, 6, 7, 10, 11, 12):
            if (out, i) != (13, 4):
                a = ptrs(14)
                a[out] = a[i]
                assert append(lib, dims(), a) == ALIAS, (out, i)
    a = ptrs(14)
    a[9] = a[8]
    assert append(lib, dims(), a) == ALIAS
    a[9] = a[8] + 64
    assert append(lib, dims(), a) == ALIAS
    assert append(lib, dims(), n=0) == gdn.GDN_OK and append(lib, dims(B=0)) == gdn.GDN_OK


def test_prefill_arguments(lib):
    check_pointers(lib, prefill, 10, (6, 8), {1: 16, 2: 16, 3: 16, 7: 16, 9: 256})
    for layer in (-1, 2):
        assert prefill(lib, dims(), layer=layer) == INV and "layer" in gdn.last_error()
    for n in (-1, 1 << 31):
        assert prefill(lib, dims(), n=n) == INV and "n_tokens" in gdn.last_error()
    for scale in (float("nan"), float("inf")):
        assert prefill(lib, dims(), scale=scale) == INV and "scale" in gdn.last_error()
    assert prefill(lib, dims(), ws=ctypes.c_uint64(16)) == INV and "workspace" in gdn.last_error()
    assert prefill(lib, dims(Hq=64), n=(1 << 31) - 1) == UNS
    for out in (7, 8, 9):
        for i in range(7):
            a = ptrs(10)
            a[out] = a[i]
            assert prefill(lib, dims(), a) == ALIAS, (out, i)
    for x, y in ((7, 8), (7, 9), (8, 9)):
        a = ptrs(10)
        a[y] = a[x]
        assert prefill(lib, dims(), a) == ALIAS
    assert prefill(lib, dims(), n=0) == gdn.GDN_OK and prefill(lib, dims(B=0)) == gdn.GDN_OK
    size = ctypes.c_uint64(0)
    assert lib.gdn_attn_prefill_workspace_size(ref(dims()), N, ctypes.byref(size)) == gdn.GDN_OK and size.value > 0
    assert lib.gdn_attn_prefill_workspace_size(ref(dims()), N, None) == INV
    assert lib.gdn_attn_prefill_workspace_size(ref(dims()), -1, ctypes.byref(size)) == INV
    assert lib.gdn_attn_prefill_workspace_size(None, N, ctypes.byref(size)) == INV
    large = kv.gdn_attn_prefill_workspace_size(dims(), 1 << 20)
    assert size.value <= large


def test_reserve_arguments(lib):
    # n_new table_in table_out len_in len_out ref_in ref_out workspace
    check_pointers(lib, reserve, 8, (), {7: 256})
    assert reserve(lib, dims(), ws=ctypes.c_uint64(16)) == INV and "workspace" in gdn.last_error()
    in_place = {(2, 1), (4, 3), (6, 5)}
    for out in (2, 4, 6, 7):
        for i in (0, 1, 3, 5):
            a = ptrs(8)
            a[out] = a[i] if (out, i) not in in_place else a[i] + 4
            assert reserve(lib, dims(), a) == ALIAS, (out, i)


def test_binding_refuses_what_is_not_on_the_device():
    d, t = dims(), torch.zeros(2, 4, 4, 64, dtype=torch.bfloat16)
    r = kv.make_rope(64, [1.0, 0.5], device="cpu")
    with pytest.raises(TypeError):
        kv.gdn_attn_rope(d, None, t, None, None, None, None, None, None, None, t, None, None)
    with pytest.raises(ValueError):
        kv.gdn_attn_rope(dims(D=128), r, t, None, None, None, None, None, None, None, t, None, None)
    with pytest.raises(ValueError):
        kv.make_rope(64, torch.zeros(33), device="cpu")
    with pytest.raises(ValueError):
        kv.make_rope(64, [1.0], q_weight=torch.zeros(32), device="cpu")
    assert r.turns.tolist() == kv.rope_turns([1.0, 0.5]).tolist()


# ---------------------------------------------------------------- turns and frequencies
def two_pi():
    """2 pi as a fraction, from Machin's formula: pi / 4 = 4 arctan(1/5) - arctan(1/239)."""
    def arctan(n, terms):
        return sum(fractions.Fraction((-1) ** k, (2 * k + 1) * n ** (2 * k + 1)) for k in range(terms))
    return 8 * (4 * arctan(5, 100) - arctan(239, 30))


def test_turns_are_right_to_the_last_bit():
    """|turns - 2^64 f / 2 pi| <= 1: the rounding, and what the two-part reciprocal of 2 pi loses (its 2^-110
    times f < 2^32 is far below 2^-64)."""
    rng = np.random.default_rng(0)
    f = np.concatenate([10000.0 ** (-np.arange(64) / 64), -10.0 ** rng.uniform(-9, 1, 40), [0.0, 1.0, math.pi, 2 * math.pi, 6.25]])
    circle, one = two_pi(), 1 << 64
    for x, turns in zip(f, kv.rope_turns(f).tolist()):
        want = fractions.Fraction(float(x)) / circle % 1 * one
        off = (turns - want) % one
        assert min(off, one - off) <= 1, x
    # large angles: the product's rest is known to 2^-53 of itself
    for x in (1e3, 123456.789, 4e9):
        off = (kv.rope_turns([x]).item() - fractions.Fraction(x) / circle % 1 * one) % one
        assert min(off, one - off) <= 1 + x * 2.0 ** -40


def test_turns_refuse_what_is_no_angle(lib):
    for bad in (float("nan"), float("inf"), 2.0 ** 32):
        with pytest.raises(gdn.GdnError):
            kv.rope_turns([0.5, bad])
    assert lib.gdn_rope_turns(None, 1, None) == INV and lib.gdn_rope_turns(None, -1, None) == INV
    assert lib.gdn_rope_turns(None, 0, None) == gdn.GDN_OK


def test_frequencies():
    f = rope.frequencies(64, 500.0)
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1.0
    assert torch.allclose(f, torch.tensor([500.0 ** (-i / 32) for i in range(32)], dtype=torch.float64))
    assert torch.equal(rope.frequencies(64, 500.0, "linear", 4.0), f / 4.0)
    g = rope.frequencies(64, 500.0, "base", 4.0)
    assert g[0] == 1.0 and abs(g[-1] / (f[-1] / 4.0) - 1.0) < 1e-12 and (g <= f).all()
    trained = 4096
    turns = f * trained / (2 * math.pi)
    for scaling in ("ramp", "bands"):
        g = rope.frequencies(64, 500.0, scaling, 8.0, trained)
        ratio = f / g
        assert (ratio >= 1.0 - 1e-12).all() and (ratio <= 8.0 + 1e-12).all() and (ratio[1:] >= ratio[:-1] - 1e-12).all()
        assert torch.allclose(ratio[turns >= 40.0], torch.ones(1, dtype=torch.float64))
        assert torch.allclose(rope.frequencies(64, 500.0, scaling, 1.0, trained), f)
    g = rope.frequencies(128, 10000.0, "bands", 8.0, trained, fast=4.0, slow=1.0)   # a pair with n turns keeps (n - 1) / 3
    f = rope.frequencies(128, 10000.0)
    n = (f * trained / (2 * math.pi)).clamp(1.0, 4.0)
    assert torch.allclose(g, f * ((n - 1) / 3 + (4 - n) / 3 / 8))
    assert rope.magnitude(1.0) == 1.0 and abs(rope.magnitude(math.e) - 1.1) < 1e-15
    assert rope.frequencies(0).shape == (0,)
    for bad in (dict(rot_dim=7), dict(rot_dim=8, scaling="other"), dict(rot_dim=8, scaling="ramp", factor=2.0),
                dict(rot_dim=8, factor=0.5), dict(rot_dim=8, base=1.0)):
        with pytest.raises(ValueError):
            rope.frequencies(**bad)


# ---------------------------------------------------------------- the oracle
def test_turn_by_hand():
    x = np.array([3.0, 0.0, 4.0, 2.0])
    quarter = [math.pi / 2]
    assert np.allclose(O.turn(x, 1, quarter), [0.0, 3.0, 4.0, 2.0])
    assert np.allclose(O.turn(x, 2, quarter, magnitude=2.0), [-6.0, 0.0, 4.0, 2.0])
    both = [math.pi / 2, math.pi]
    assert np.allclose(O.turn(x, 1, both), [-4.0, 0.0, 3.0, -2.0])          # pairs (0, 2) and (1, 3)
    assert np.allclose(O.turn(x, 1, both, interleaved=True), [0.0, 3.0, -4.0, -2.0])
    rms = math.sqrt(29 / 4)
    assert np.allclose(O.turn(x, 0, both, weight=[0, 1, 2, 3], weight_offset=1.0), x / rms * [1, 2, 3, 4])


def test_turn_keeps_what_a_rotation_keeps():
    """Norms, and products of queries and keys as a function of the distance alone."""
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(2, 16))
    f = 10000.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        dots = [O.turn(q, p + 5, f, inter) @ O.turn(k, p, f, inter) for p in (0, 7, 1000, 123456)]
        assert np.allclose(dots, dots[0])
        assert np.isclose(np.linalg.norm(O.turn(q, 99, f, inter)), np.linalg.norm(q))
    half = O.turn(q, 3, f)
    shuffled = np.stack([q[:8], q[8:]], 1).ravel()                           # the two layouts, one into the other
    assert np.allclose(O.turn(shuffled, 3, f, True).reshape(8, 2).T.ravel(), half)


def test_window_and_append_agree_and_positions_follow_the_tree():
    rng = np.random.default_rng(1)
    parent = [[-1, 0, 0, 2, -1]]
    assert O.window_positions([7, 100], [1], parent, 1, 5).tolist() == [[107, 108, 108, 109, 107]]
    assert O.window_positions([7, 100], None, None, 1, 3).tolist() == [[7, 8, 9]]
    f = [1.0, 0.3]
    q, k, v = rng.normal(size=(5, 2, 8)), rng.normal(size=(5, 1, 8)), rng.normal(size=(5, 1, 8))
    cache = np.zeros((2, 4, 1, 8))
    table, lens = np.array([[1, 0], [-1, -1]]), np.array([7, 3])
    out, ck, cv = O.append([0, 5], q, k, v, cache, cache, table, lens, [1], np.zeros_like(q), None, None, [1.0] * 8, radians=f)
    pos = O.window_positions([2, 3], [1], None, 1, 5)
    assert np.allclose(out, O.window(q[None], pos, None, None, radians=f)[0])
    want = O.window(k[None], pos, None, [1.0] * 8, radians=f)[0]
    assert np.allclose(np.concatenate([ck[1], ck[0]])[2:7], want) and np.allclose(np.concatenate([cv[1], cv[0]])[2:7], v)
    assert (ck[1, :2] == 0).all() and (ck[0, 3] == 0).all()


def test_reserve_oracle_by_hand():
    table, lens, cnt = np.array([[2, -1, -1], [-1, -1, -1]]), np.array([1, 0]), np.array([0, 7, 1, 0, 0])
    t, n, r = O.reserve([2, 3], table, lens, cnt, 2)
    assert t.tolist() == [[2, 0, -1], [3, 4, -1]] and n.tolist() == [3, 3] and r.tolist() == [1, 7, 1, 1, 1]
    t, n, r = O.reserve([4, 3], table, lens, cnt, 2)      # the second finds two pages taken, and one of two
    assert t.tolist() == [[2, 0, 3], [-1, -1, -1]] and n.tolist() == [5, 0] and r.tolist() == [1, 7, 1, 1, 0]


def test_prefill_oracle_against_a_masked_softmax():
    rng = np.random.default_rng(2)
    ck, cv = rng.normal(size=(2, 6, 4, 2, 8))
    table, lens = np.array([[3, 1, -1], [0, 5, 2]]), np.array([7, 10])
    q = rng.normal(size=(4, 4, 8))
    for causal in (False, True):
        out, lse = O.attention([0, 3, 3], q, ck, cv, table, lens, [1, -1], causal, 0.4)
        assert np.isnan(out[3]).all()
        k, v = (np.concatenate([c[[0, 5, 2]].reshape(-1, 2, 8)[:10], c[[3, 1]].reshape(-1, 2, 8)[:7]]) for c in (ck, cv))
        mask = np.tril(np.ones((3, 17)), 14) > 0 if causal else np.ones((3, 17)) > 0
        for h in range(4):
            x = np.where(mask, 0.4 * q[:3, h] @ k[:, h // 2].T, -np.inf)
            w = np.exp(x) / np.exp(x).sum(1, keepdims=True)
            assert np.allclose(out[:3, h], w @ v[:, h // 2]) and np.allclose(lse[:3, h], np.log(np.exp(x).sum(1)))
    out, lse = O.attention([0, 3], q[:3], ck, cv, table, np.array([1, 0]), None, True, 1.0)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(out[2, 0], cv[3, 0, 0])


def test_cache_calls_on_sequences_and_prefixes(monkeypatch):
    """Prompts of sequences take their prefixes along, and those of prefixes have none.  One call on both kinds, whose
    prefixes are no slice, is refused; pages for all slots at once fit the cache's workspace."""
    build.build_library()
    seen = []
    monkeypatch.setattr(kv, "gdn_kv_append", lambda *args: seen.append(args[-3]))
    monkeypatch.setattr(kv, "gdn_attn_prefill", lambda *args: seen.append(args[8]))
    c = PagedCache.create(40, 1, 2, 1, 64, 16, n_pages=20, max_pages=4, n_prefixes=60, device="cpu")
    c.prefix_of.copy_(torch.arange(40, dtype=torch.int32) + 40)
    rows = torch.zeros(3, 2, 64, dtype=torch.bfloat16)

    def both(n, slot0):
        cu = torch.zeros(n + 1, dtype=torch.int32)
        c.append_layer(0, None, cu, rows, rows[:, :1], rows[:, :1], rows, slot0=slot0)
        c.attend_prefill(0, cu, rows, torch.empty_like(rows), slot0=slot0)
        return seen[-2:]

    for n, slot0 in ((40, 0), (3, 37), (1, 0)):
        assert all(p.tolist() == list(range(40 + slot0, 40 + slot0 + n)) for p in both(n, slot0))
    assert both(60, 40) == [None, None] and both(1, 99) == [None, None]
    for n, slot0 in ((41, 0), (2, 39), (100, 0)):
        with pytest.raises(ValueError, match="prefixes"):
            both(n, slot0)
    assert c.pool_workspace.numel() >= kv.gdn_kv_workspace_size(c._dims(100))
