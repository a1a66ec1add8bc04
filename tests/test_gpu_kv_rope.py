"""Norms and rotation of windows, reserve, and append of packed tokens, against the float64 oracle.

Tolerances.  Everything is f32 until one rounding, at most u = eps / 2 of the type.  A norm sums D <= 128
squares: its relative error is at most 128 * 2^-24 / 2 and two units of the reciprocal root, 4.1e-6; the
angle is off by at most 2^-25 half turns, 1e-7, sine and cosine by 2^-23 each, and the two products and their
sum by 3 * 2^-24 of what is summed.  Hence |out - ref| <= u |ref| + 6e-6 M, M = magnitude (|a| + |b|) over the pair
(|x| where nothing is rotated); f16 adds half of its smallest step, 2^-25."""
import numpy as np
import pytest
import torch

from kv_util import ROUND, Pool, f64, i32, random_trees
from oracle import prompt_oracle as O
from speculative_decode_verify_gdn_gb300 import gdn, kv, rope
from speculative_decode_verify_gdn_gb300.build import build_library

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    build_library()
    kv.load_library()
    gdn.gdn_device_status(clear=True)
    yield
    assert gdn.gdn_device_status(clear=True) == 0


class Turning:
    """A rotation on the device and as the oracle takes it."""

    def __init__(self, seed, D, rot, inter=False, norm=True, magnitude=1.0, offset=0.0, base=10000.0):
        rng = np.random.default_rng(seed)
        self.radians = rope.frequencies(rot, base).numpy()
        self.w = [torch.from_numpy(rng.normal(1.0 - offset, 0.2, D)).float() if norm else None for _ in range(2)]
        self.how = dict(radians=self.radians, interleaved=inter, magnitude=magnitude, eps=1e-6, weight_offset=offset)
        self.rope = kv.make_rope(D, self.radians, inter, magnitude, *(None if w is None else w.cuda() for w in self.w),
                                 eps=1e-6, weight_offset=offset)
        self.host = [None if w is None else w.double().numpy() for w in self.w]

    def bound(self, x, weight):
        """M of the tolerance for heads x [.., D]."""
        D = x.shape[-1]
        y = np.abs(x)
        if weight is not None:
            y = np.abs(x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * (self.how["weight_offset"] + weight))
        half = len(self.radians)
        m = y.copy()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if self.how["interleaved"] else (i, i + half)
            m[..., a] = m[..., b] = abs(self.how["magnitude"]) * (y[..., a] + y[..., b])
        assert m.shape[-1] == D
        return m


def close(got, want, m, dtype):
    bad = np.abs(f64(got) - want) > ROUND[dtype] * np.abs(want) + 6e-6 * m + (2.0 ** -25 if dtype == HF else 0.0)
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(f64(got) - want).max())


def gauss(seed, *shape, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def projection(seed, B, K, Hq, Hkv, D, dtype, gate):
    wide = 2 if gate else 1
    x = gauss(seed, B, K, (Hq * wide + 2 * Hkv) * D, dtype=dtype)
    q, k, v = x.split([Hq * wide * D, Hkv * D, Hkv * D], -1)
    return x, q.view(B, K, Hq, wide * D)[..., :D], k.view(B, K, Hkv, D), v.view(B, K, Hkv, D)


def window_case(seed, B, K, Hq, Hkv, D, dtype=BF, rot=None, gate=False, ragged=False, tree=False, prefixes=0, lens=None,
                positions=None, slot0=0, in_place=False, **turning):
    rng = np.random.default_rng(seed)
    t = Turning(seed, D, D if rot is None else rot, **turning)
    x, q, k, v = projection(seed, B, K, Hq, Hkv, D, dtype, gate)
    n_slots = slot0 + B + prefixes
    lens = rng.integers(0, 1000, n_slots) if lens is None else np.asarray(lens)
    pre = None if not prefixes else slot0 + B + rng.integers(-1, prefixes, B) if prefixes > 1 else np.full(B, slot0 + B)
    if pre is not None:
        pre = np.where(pre < slot0 + B, -1, pre)
    win = rng.integers(0, K + 1, B) if ragged else None
    par = random_trees(rng, B, K) if tree else None
    if ragged:
        for b in range(B):
            x[b, int(win[b]):] = NAN
    want_x = [np.nan_to_num(f64(y)) for y in (q, k, v)]
    d = kv.make_kv_dims(B, K, Hq, Hkv, D, 16, 1, 1 << 26, n_slots=n_slots, slot0=slot0, dtype=dtype,
                        q=q if in_place else None, win=k if in_place else None)
    outs = [q, k, v] if in_place else [torch.full((B, K, h, D), NAN, dtype=dtype, device="cuda") for h in (Hq, Hkv, Hkv)]
    opt = [None if y is None else i32(y) for y in (pre, win, par, positions)]
    kv.gdn_attn_rope(d, t.rope, q, k, v, None if positions is not None else i32(lens), *opt, *outs)
    pos = O.window_positions(lens, pre, par, B, K, slot0) if positions is None else positions
    for got, y, w in zip(outs[:2], want_x[:2], t.host):
        close(got, O.window(y, pos, win, w, **t.how), t.bound(y, w), dtype)
    live = np.ones((B, K)) if win is None else (np.arange(K)[None] < win[:, None])
    assert np.array_equal(f64(outs[2]), want_x[2] * live[:, :, None, None])
    return outs


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (64, 0), (64, 48), (128, 128), (128, 32), (128, 16), (128, 112)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_parts_of_the_head_in_both_layouts(D, rot, inter, dtype):
    window_case(1, 3, 4, 6, 2, D, dtype, rot, inter=inter)
    window_case(2, 2, 3, 3, 1, D, dtype, rot, inter=inter, norm=False, magnitude=1.3)


@pytest.mark.parametrize("B,K,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 16, 2), (1, 16, 5, 5), (7, 3, 12, 3), (700, 2, 2, 1), (90, 16, 1, 1)])
@pytest.mark.parametrize("gate", [False, True])
def test_sizes(B, K, Hq, Hkv, gate):
    window_case(3, B, K, Hq, Hkv, 64, gate=gate, offset=1.0)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("tree", [False, True])
def test_trees_padding_and_prefixes(dtype, tree):
    for K in (1, 2, 7, 16):
        window_case(4 + K, 9, K, 4, 2, 128, dtype, ragged=True, tree=tree, prefixes=3, slot0=2)
        window_case(5 + K, 5, K, 4, 2, 64, dtype, tree=tree, prefixes=1, gate=True)


def test_positions_up_to_the_longest_slots():
    """Angles stay exact where a 32-bit product of position and frequency is off by radians: the oracle's own
    are taken modulo a turn in float64, off by 2^-53 of 2^31 radians."""
    top = (1 << 30) - 1
    window_case(6, 5, 4, 4, 2, 128, lens=[0, 1 << 20, 123456789, (1 << 29) + 1, top - 3], norm=False)
    window_case(7, 2, 3, 4, 2, 64, lens=[top, 0, top], prefixes=1, dtype=HF)   # a prefix and a slot of 2^30 tokens
    far = np.array([[0, -1, -5], [(1 << 31) - 1, -(1 << 31), 1000003]])
    window_case(8, 2, 3, 4, 2, 64, positions=far, inter=True, dtype=HF)


@pytest.mark.parametrize("ragged", [False, True])
def test_in_place_in_the_projection(ragged):
    window_case(9, 5, 4, 6, 2, 64, in_place=True, ragged=ragged, tree=True)
    window_case(10, 333, 16, 6, 2, 128, in_place=True, ragged=ragged, rot=64)


def test_parts_alone():
    """Queries alone, keys alone, values alone give what they give together."""
    B, K, Hq, Hkv, D = 3, 2, 4, 2, 64
    t = Turning(11, D, 32)
    _, q, k, v = projection(11, B, K, Hq, Hkv, D, BF, False)
    d = kv.make_kv_dims(B, K, Hq, Hkv, D, 16, 1, 64)
    lens = i32([5, 0, 100])
    whole = [torch.empty((B, K, h, D), dtype=BF, device="cuda") for h in (Hq, Hkv, Hkv)]
    kv.gdn_attn_rope(d, t.rope, q, k, v, lens, None, None, None, None, *whole)
    for i, x in enumerate((q, k, v)):
        out = torch.empty_like(whole[i])
        ins, outs = [None] * 3, [None] * 3
        ins[i], outs[i] = x, out
        kv.gdn_attn_rope(d, t.rope, *ins, lens, None, None, None, None, *outs)
        assert torch.equal(out, whole[i])


def test_heads_before_tokens_and_other_strides():
    """Inputs whose heads lie further apart than their tokens, and outputs within wider rows."""
    B, K, Hq, Hkv, D = 3, 4, 4, 2, 64
    t = Turning(12, D, 64)
    q = gauss(12, Hq, B, K, D).permute(1, 2, 0, 3)
    k, v = (gauss(13 + i, Hkv, B, K, D).permute(1, 2, 0, 3) for i in range(2))
    lens = i32([5, 0, 100])
    ref = [torch.empty((B, K, h, D), dtype=BF, device="cuda") for h in (Hq, Hkv, Hkv)]
    d = kv.make_kv_dims(B, K, Hq, Hkv, D, 16, 1, 64)
    kv.gdn_attn_rope(d, t.rope, q.contiguous(), k.contiguous(), v.contiguous(), lens, None, None, None, None, *ref)
    wide = torch.full((B, K, (Hq + 2 * Hkv + 3) * D), 7.0, dtype=BF, device="cuda")
    qo = wide[..., D:(1 + Hq) * D].unflatten(-1, (Hq, D))
    ko = wide[..., (1 + Hq) * D:(1 + Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    vo = wide[..., (2 + Hq + Hkv) * D:(2 + Hq + 2 * Hkv) * D].unflatten(-1, (Hkv, D))
    d = kv.make_kv_dims(B, K, Hq, Hkv, D, 16, 1, 64, q=qo, win=ko)
    kv.gdn_attn_rope(d, t.rope, q, k, v, lens, None, None, None, None, qo, ko, vo)
    assert all(torch.equal(a, b) for a, b in zip((qo, ko, vo), ref))
    for lo, hi in ((0, 1), (1 + Hq + Hkv, 2 + Hq + Hkv), (2 + Hq + 2 * Hkv, 3 + Hq + 2 * Hkv)):
        assert (wide[..., lo * D:hi * D] == 7.0).all()
    with pytest.raises(ValueError):
        kv.gdn_attn_rope(d, t.rope, q.contiguous(), k, v, lens, None, None, None, None, q, ko, vo)
    with pytest.raises(ValueError):
        kv.gdn_attn_rope(d, t.rope, q, k, v.contiguous(), lens, None, None, None, None, qo, ko, vo)
    with pytest.raises(ValueError):
        kv.gdn_attn_rope(d, t.rope, q.transpose(0, 1).contiguous().transpose(0, 1), k, v, lens, None, None, None, None, qo, ko, vo)


def test_status_of_windows():
    """Lengths, windows, prefixes and parents that are out of range are reported, and read as the contract says."""
    B, K, D = 3, 4, 64
    t = Turning(14, D, 64)
    _, q, k, v = projection(14, B, K, 2, 1, D, BF, False)
    d = kv.make_kv_dims(B, K, 2, 1, D, 16, 1, 64, n_slots=4)
    outs = [torch.empty((B, K, h, D), dtype=BF, device="cuda") for h in (2, 1, 1)]

    def run(lens=(5, 6, 7, 8), pre=(-1, 3, 3), win=(4, 4, 4), par=None):
        par = [[-1, 0, 0, 1]] * B if par is None else par
        kv.gdn_attn_rope(d, t.rope, q, k, v, i32(lens), i32(pre), i32(win), i32(par), None, *outs)
        return gdn.gdn_device_status(clear=True), [o.clone() for o in outs]

    ok, ref = run()
    assert ok == 0
    for bad, good, bit in ((dict(lens=(-1, 6, 7, 8)), dict(lens=(0, 6, 7, 8)), kv.DEVERR_KV_LEN),
                           (dict(lens=(5, 1025, 7, 8)), dict(lens=(5, 0, 7, 8)), kv.DEVERR_KV_LEN),
                           (dict(pre=(4, 3, -2)), dict(pre=(-1, 3, -1)), kv.DEVERR_KV_SLOT),
                           (dict(win=(5, -1, 4)), dict(win=(4, 0, 4)), kv.DEVERR_KV_WINDOW),
                           (dict(par=[[-1, 0, 2, 1]] * B), dict(par=[[-1, 0, -1, 1]] * B), gdn.DEVERR_TREE_PARENT)):
        status, got = run(**bad)
        assert status == bit, bad
        status, want = run(**good)
        assert status == 0 and all(torch.equal(a, b) for a, b in zip(got, want)), bad


# ---------------------------------------------------------------- reserve
def reserve(pool, n_new, B, slot0=0, in_place=False, ws_fill=255):
    d = pool.dims(B, slot0=slot0)
    books = [i32(x) for x in (pool.table, pool.lens, pool.ref)]
    outs = books if in_place else [torch.full_like(x, -77) for x in books]
    ws = kv.alloc_kv_workspace(d)
    ws.fill_(ws_fill)
    kv.gdn_kv_reserve(d, i32(n_new), books[0], outs[0], books[1], outs[1], books[2], outs[2], ws)
    got = [x.cpu().numpy() for x in outs]
    want = O.reserve(n_new, pool.table, pool.lens, pool.ref, pool.ps, slot0)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    return got


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,new,spare", [
    ([0], [1], 1), ([700], [4], 5), ([15, 16, 17, 0], [1, 1, 1, 0], 10), ([5, 0, 33, 16], [300, 1, 0, 17], 40),
    ([5, 0, 33, 16], [300, 1, 0, 17], 21), ([5, 0, 33, 16], [300, 1, 0, 17], 0), ([3] * 600, list(range(600)), 20000),
    ([3] * 600, list(range(600)), 2000), ([100] * 1500, [40] * 1500, 6000)])
def test_reserve(lens, new, spare, in_place):
    """One sequence, sequences around a page, pools that run out, batches of more than one step and pools that a
    cluster shares."""
    pool = Pool(20, lens, layers=1, Hkv=1, spare=spare, max_pages=max(-(-(n + m) // 16) for n, m in zip(lens, new)) + 1)
    grown = reserve(pool, new, len(lens), in_place=in_place)[1]
    needs = np.cumsum([-(-(n + m) // 16) - -(-n // 16) for n, m in zip(lens, new)])
    full = bool((needs > spare).any())
    assert gdn.gdn_device_status(clear=True) == (kv.DEVERR_KV_FULL if full else 0)
    assert full or np.array_equal(grown, np.add(lens, new))


def test_reserve_in_a_part_of_the_slots():
    pool = Pool(21, [40, 5, 16, 0, 33], spare=30, max_pages=12)
    reserve(pool, [100, 1, 64], 3, slot0=1)
    reserve(pool, [100, 1, 64], 3, slot0=1, in_place=True)
    reserve(pool, [], 0)


def test_reserve_where_it_cannot():
    """Shared last pages, rows without columns, numbers out of range: those sequences alone stay as they are."""
    pool = Pool(22, [40, 32, 16, 5, 7], spare=30, max_pages=4)
    pool.ref[pool.table[0, 2]] = 2                        # the first one's last page is shared
    reserve(pool, [1, 1, 49, 3, 0], 5)
    assert gdn.gdn_device_status(clear=True) == kv.DEVERR_KV_SHARED | kv.DEVERR_KV_FULL
    pool.ref[pool.table[0, 2]] = 1
    for bad in (-1, (1 << 30) + 1, (1 << 31) - 1, -(1 << 31)):
        d = pool.dims(5)
        books = [i32(x) for x in (pool.table, pool.lens, pool.ref)]
        kv.gdn_kv_reserve(d, i32([1, bad, 1, 0, 2]), books[0], books[0], books[1], books[1], books[2], books[2],
                          kv.alloc_kv_workspace(d))
        assert gdn.gdn_device_status(clear=True) == kv.DEVERR_KV_LEN
        for g, w in zip(books, O.reserve([1, 0, 1, 0, 2], pool.table, pool.lens, pool.ref, pool.ps)):
            assert np.array_equal(g.cpu().numpy(), w)
    lens, table = pool.lens.copy(), pool.table.copy()
    lens[1], table[3, 0] = -4, 1 << 20
    d = pool.dims(5)
    books = [i32(x) for x in (table, lens, pool.ref)]
    kv.gdn_kv_reserve(d, i32([1, 1, 1, 1, 1]), books[0], books[0], books[1], books[1], books[2], books[2], kv.alloc_kv_workspace(d))
    assert gdn.gdn_device_status(clear=True) == kv.DEVERR_KV_LEN | kv.DEVERR_KV_PAGE
    assert books[1].tolist() == [41, -4, 17, 5, 8]


def test_reserve_refers_to_what_commit_would_take():
    """The pages and lengths are those of a commit of as many tokens."""
    lens, new = [15, 16, 0, 100, 48], [3, 16, 1, 0, 33]
    pool = Pool(23, lens, layers=2, spare=12, max_pages=9)
    got = reserve(pool, new, 5)
    d = pool.dims(5, K=33)
    win = [torch.zeros((2, 5, 33, pool.Hkv, pool.D), dtype=BF, device="cuda") for _ in range(2)]
    books = [i32(x) for x in (pool.table, pool.lens, pool.ref)]
    kv.gdn_kv_commit(d, i32(new), None, *win, pool.k, pool.v, books[0], books[0], books[1], books[1], books[2], books[2],
                     kv.alloc_kv_workspace(d))
    for g, w in zip(got, books):
        assert np.array_equal(g, w.cpu().numpy())


# ---------------------------------------------------------------- append
def append_case(seed, new, before, Hq, *, prefixes=(), pre=None, rot=None, gate=False, spare_rows=0, positions=False,
                layer=0, slot0=0, in_place=False, with_q=True, turning={}, **pool_args):
    new, before = np.asarray(new), np.asarray(before)
    B = len(new)
    pool = Pool(seed, [7] * slot0 + list(new + before) + list(prefixes), **pool_args)
    D, Hkv, dtype = pool.D, pool.Hkv, pool.dtype
    t = Turning(seed, D, D if rot is None else rot, **turning)
    cu = np.concatenate([[0], np.cumsum(new)])
    n = int(cu[-1]) + spare_rows
    x, q, k, v = (y[0] for y in projection(seed, 1, n, Hq, Hkv, D, dtype, gate))
    x[int(cu[-1]):] = NAN
    src = [np.nan_to_num(f64(y)) for y in (q, k, v)]
    pos = pool.rng.integers(0, 5000, n) if positions else None
    q_out = q if in_place else torch.full((n, Hq, D), 3.0, dtype=dtype, device="cuda")
    d = kv.make_kv_dims(B, 1, Hq, Hkv, D, pool.ps, pool.n_pages, pool.max_pages, len(pool.lens), slot0, pool.layers, dtype,
                        cache=pool.k, q=q if in_place else None)
    kept = [y.clone() for y in (pool.k, pool.v, q_out)]
    kv.gdn_kv_append(d, layer, t.rope, i32(cu), q if with_q else None, k, v, None if pos is None else i32(pos), pool.k, pool.v,
                     i32(pool.table), i32(pool.lens), None if pre is None else i32(pre), q_out if with_q else None)
    want_q, want_k, want_v = O.append(cu, src[0], src[1], src[2], f64(kept[0][layer]), f64(kept[1][layer]), pool.table, pool.lens,
                                      pre, np.zeros((n, Hq, D)), pos, *t.host, slot0=slot0, **t.how)
    # what the append is to write, and only that
    mark = O.append(cu, src[0], np.ones_like(src[1]), np.ones_like(src[1]), np.zeros(pool.k[0].shape), np.zeros(pool.k[0].shape),
                    pool.table, pool.lens, pre, np.zeros((n, Hq, D)), pos, None, None, slot0=slot0, radians=[])[1] > 0
    bound_k = np.zeros(pool.k[0].shape)
    bound_k[mark] = O.append(cu, src[0], t.bound(src[1], t.host[1]), src[2], bound_k, bound_k, pool.table, pool.lens, pre,
                             np.zeros((n, Hq, D)), pos, None, None, slot0=slot0, radians=[])[1][mark]
    got_k, got_v = f64(pool.k[layer]), f64(pool.v[layer])
    assert np.array_equal(got_v[mark], want_v[mark])
    close(pool.k[layer].double()[torch.from_numpy(mark).cuda()], want_k[mark], bound_k[mark], dtype)
    for got, was in ((got_k, kept[0]), (got_v, kept[1])):
        assert np.array_equal(got[~mark], f64(was[layer])[~mark], equal_nan=True)
    for other in range(pool.layers):
        if other != layer:
            assert torch.equal(pool.k[other].view(torch.int16), kept[0][other].view(torch.int16))
    if with_q:
        m = int(cu[-1])
        close(q_out[:m], want_q[:m], t.bound(src[0][:m], t.host[0]), dtype)
        assert torch.equal(q_out[m:].contiguous().view(torch.int16), kept[2][m:].contiguous().view(torch.int16))


@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64)])
@pytest.mark.parametrize("ps", [16, 48, 112])
@pytest.mark.parametrize("order", ["nhd", "hnd", "mixed"])
def test_append_to_pages_of_any_size_and_order(dtype, D, ps, order):
    append_case(30, [1, 17, 0, 130, 48], [0, 15, 33, 100, 0], 4, dtype=dtype, D=D, ps=ps, order=order, layers=2, layer=1)


@pytest.mark.parametrize("new,before", [([1], [0]), ([1], [500]), ([1] * 40, list(range(40))), ([0, 0, 3, 0], [5, 0, 1, 9]),
                                        ([1, 0] * 600, [3] * 1200), ([1500], [7]), ([0], [3])])
def test_append_sizes(new, before):
    """Single tokens, batches of more than 32 and 1024 sequences, empty ones, whole prompts."""
    append_case(31, new, before, 3, Hkv=1, D=64, spare_rows=5)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_append_behind_prefixes(gate, inter):
    append_case(32, [5, 40, 1, 7], [20, 0, 31, 2], 6, prefixes=[50, 1000], pre=[6, -1, 7, 6], slot0=2, gate=gate, rot=32,
                turning=dict(inter=inter, magnitude=1.2, offset=1.0))
    append_case(33, [5, 40, 1, 7], [20, 0, 31, 2], 6, prefixes=[50], pre=[4, 4, -1, 4], positions=True, gate=gate,
                turning=dict(inter=inter, norm=False), D=128)


def test_append_in_place_and_without_queries():
    append_case(34, [5, 40, 100], [20, 0, 31], 6, in_place=True, spare_rows=3, D=128)
    append_case(35, [5, 40, 100], [20, 0, 31], 6, with_q=False, rot=0)


def test_status_of_appends():
    """What is out of range is reported, and only what belongs to it is left out."""
    pool = Pool(36, [20, 40, 30, 9], ps=16, Hkv=1, D=64)
    t = Turning(36, 64, 64)
    N = 30
    q, k, v = gauss(36, N, 2, 64), gauss(37, N, 1, 64), gauss(38, N, 1, 64)
    d = pool.dims(3, 1, 2)
    clean = [pool.k.clone(), pool.v.clone()]

    def run(cu=(0, 10, 15, 30), lens=(20, 40, 30, 9), table=pool.table, pre=(3, -1, -1)):
        kc, vc = clean[0].clone(), clean[1].clone()
        out = torch.zeros_like(q)
        kv.gdn_kv_append(d, 0, t.rope, i32(cu), q, k, v, None, kc, vc, i32(table), i32(lens), i32(pre), out)
        return gdn.gdn_device_status(clear=True), kc.nan_to_num(), vc.nan_to_num(), out

    status, kc, vc, out = run()
    assert status == 0
    table = pool.table.copy()
    table[1, 2] = -1                                       # holds the second one's last 8 tokens
    status, k2, v2, o2 = run(table=table)
    assert status == kv.DEVERR_KV_PAGE and torch.equal(o2, out)
    last = int(pool.table[1, 2])
    assert torch.equal(k2[0, last], clean[0][0, last].nan_to_num())
    keep = torch.arange(pool.n_pages, device="cuda") != last
    assert torch.equal(k2[0, keep], kc[0, keep]) and torch.equal(v2[0, keep], vc[0, keep])
    status, k2, v2, o2 = run(lens=(9, 40, 30, 9))          # ten tokens in a slot of nine
    assert status == kv.DEVERR_KV_LEN
    assert (o2[:10] == 0).all() and torch.equal(o2[10:], out[10:])
    status, k2, v2, o2 = run(lens=(20, 40, -3, 9))
    assert status == kv.DEVERR_KV_LEN and (o2[15:] == 0).all()
    status, _, _, o2 = run(pre=(7, -1, -2))
    assert status == kv.DEVERR_KV_SLOT
    for cu in ((0, 10, 15, 31), (1, 10, 15, 30), (0, 15, 10, 30), (0, -5, 15, 30)):
        status, k2, v2, _ = run(cu=cu)
        assert status & gdn.DEVERR_SEQLENS and not status & ~(gdn.DEVERR_SEQLENS | kv.DEVERR_KV_LEN), cu
