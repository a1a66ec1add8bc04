"""Attention of verify windows over the paged cache against the float64 oracle.

Tolerances.  With u the rounding of the 16-bit type (2^-8 bf16, 2^-11 f16), an output element is
off by at most u * sum_j w_j |v_j| for the rounded probabilities and u |o| for its own rounding.
Scores are f32 sums of D <= 128 products: with |q| of a few units their error stays below
128 * 2^-24 * scale * sum |q_i k_i| <= 1e-4, which moves every weight by that fraction at most.
Hence |out - ref| <= u (A + |ref|) + 2e-4 A with A = sum_j w_j |v_j|, and |lse - ref| <= 1e-4."""
import numpy as np
import pytest
import torch

from kv_util import ROUND, Pool, f64, i32, random_trees
from oracle import kv_oracle as O
from speculative_decode_verify_gdn_gb300 import gdn, kv
from speculative_decode_verify_gdn_gb300.build import build_library

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    build_library()
    kv.load_library()
    gdn.gdn_device_status(clear=True)
    yield
    assert gdn.gdn_device_status(clear=True) == 0


def window(pool, B, K, Hq, win_len=None, q_scale=2.0):
    """q, k_win, v_win with NaN at padding tokens."""
    q, k, v = pool.gauss((B, K, Hq, pool.D), q_scale), pool.gauss((B, K, pool.Hkv, pool.D)), pool.gauss((B, K, pool.Hkv, pool.D))
    if win_len is not None:
        for b in range(B):
            for x in (q, k, v):
                x[b, int(win_len[b]):] = float("nan")
    return q, k, v


def attend(pool, B, K, Hq, q, k, v, prefix_of=None, win_len=None, parent=None, layer=0, slot0=0, scale=None,
           lse=True, dims=None):
    dims = dims or pool.dims(B, K, Hq, slot0)
    out = torch.full((B, K, Hq, pool.D), float("nan"), dtype=pool.dtype, device="cuda")
    ls = torch.full((B, K, Hq), float("nan"), dtype=torch.float32, device="cuda") if lse else None
    opt = [None if x is None else i32(x) for x in (prefix_of, win_len, parent)]
    ws = kv.alloc_attn_workspace(dims)
    ws.fill_(255)
    kv.gdn_attn_verify(dims, layer, q, k, v, pool.k, pool.v, i32(pool.table), i32(pool.lens), *opt,
                       pool.D ** -0.5 if scale is None else scale, out, ls, ws)
    return out, ls


def check(pool, B, K, Hq, q, k, v, out, lse, prefix_of=None, win_len=None, parent=None, layer=0, slot0=0, scale=None):
    zero = lambda t: np.nan_to_num(f64(t))  # noqa: E731  (the oracle reads no NaN place, but multiplies by rows)
    args = (f64(pool.k[layer]), f64(pool.v[layer]), pool.table, pool.lens, prefix_of, win_len, parent,
            pool.D ** -0.5 if scale is None else scale, slot0)
    ref, ref_lse = O.attention(zero(q), zero(k), zero(v), *args)
    mag, _ = O.attention(zero(q), zero(k), np.abs(zero(v)), args[0], np.abs(args[1]), *args[2:])
    u = ROUND[pool.dtype]
    got = f64(out)
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > u * (mag + np.abs(ref)) + 2e-4 * mag
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - ref).max())
    if lse is not None:
        empty = np.isinf(ref_lse)
        got = f64(lse)
        assert np.array_equal(np.isneginf(got), empty)
        assert np.abs(got[~empty] - ref_lse[~empty]).max(initial=0) <= 1e-4


def run_case(seed, lens, B, K, Hq, prefix_of=None, ragged=False, tree=False, slot0=0, layer=0, **pool_args):
    pool = Pool(seed, lens, **pool_args)
    win = pool.rng.integers(0, K + 1, B) if ragged else None
    par = random_trees(pool.rng, B, K) if tree else None
    q, k, v = window(pool, B, K, Hq, win)
    out, lse = attend(pool, B, K, Hq, q, k, v, prefix_of, win, par, layer, slot0)
    check(pool, B, K, Hq, q, k, v, out, lse, prefix_of, win, par, layer, slot0)
    return pool, out, lse


LENS = [0, 1, 15, 16, 17, 111, 112, 113, 127, 128, 129, 255, 256, 300]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("K", [1, 4, 16])
def test_own_lengths_around_the_tile(D, dtype, K):
    run_case(1, LENS, len(LENS), K, 4, D=D, dtype=dtype)


@pytest.mark.parametrize("ps", [16, 32, 48, 64, 80, 128, 256, 1024])
@pytest.mark.parametrize("order", ["nhd", "hnd", "mixed"])
def test_page_sizes_and_orders(ps, order):
    run_case(2, [0, 1, ps - 1, ps, ps + 1, 130, 200, 333], 6, 5, 4, prefix_of=[7, 7, -1, 6, 6, 6], ps=ps, order=order, D=128)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (6, 2), (5, 1), (24, 3), (20, 1), (64, 2)])
@pytest.mark.parametrize("K", [1, 7, 16])
def test_heads(Hq, Hkv, K):
    run_case(3, [40, 0, 150, 200], 3, K, Hq, prefix_of=[3, 3, 3], Hkv=Hkv, D=64, ragged=True)


@pytest.mark.parametrize("plen", [0, 1, 16, 127, 128, 129, 700])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64)])
def test_prefix_lengths(plen, dtype, D):
    run_case(4, [3, 90, 0, 17, 260, plen], 5, 3, 8, prefix_of=[5] * 5, Hkv=2, D=D, dtype=dtype)


def test_many_sequences_on_one_prefix_fill_row_blocks():
    """Row counts of the shared pass around 128 and 256: B K G = 126, 128, 130, 256, 258, 400."""
    for B, K, G in ((21, 3, 2), (16, 8, 1), (13, 5, 2), (16, 16, 1), (43, 3, 2), (25, 16, 1)):
        run_case(5 + B, list(range(B)) + [140], B, K, G, prefix_of=[B] * B, Hkv=1, D=64)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_ragged_windows_trees_and_mixed_prefixes(tree, dtype):
    """Runs of equal prefixes, sequences without one, a prefix met again later, a sequence's own slot
    as another's prefix, windows of length 0."""
    lens = [5, 77, 0, 130, 128, 31, 64, 1, 260, 40]
    run_case(6, lens, 8, 16, 4, prefix_of=[8, 8, -1, 9, 8, 0, 0, -1], ragged=True, tree=tree, dtype=dtype, D=128)


def test_only_the_window():
    """Nothing cached anywhere: every row sees its ancestors alone."""
    run_case(7, [0, 0, 0], 3, 16, 2, tree=True, max_pages=1, n_pages=1)


def test_no_window_token_at_all():
    pool = Pool(8, [20, 300, 50])
    q, k, v = window(pool, 3, 4, 4, [0, 0, 0])
    out, lse = attend(pool, 3, 4, 4, q, k, v, prefix_of=[1, 1, 1], win_len=[0, 0, 0])
    assert torch.equal(out, torch.zeros_like(out)) and torch.isneginf(lse).all()


def test_later_slots_layers_and_no_lse():
    pool = Pool(9, [10, 20, 200, 33, 150], layers=3, D=128)
    q, k, v = window(pool, 2, 4, 4)
    for layer in range(3):
        out, lse = attend(pool, 2, 4, 4, q, k, v, prefix_of=[4, 0], layer=layer, slot0=2)
        check(pool, 2, 4, 4, q, k, v, out, lse, prefix_of=[4, 0], layer=layer, slot0=2)
        out2, _ = attend(pool, 2, 4, 4, q, k, v, prefix_of=[4, 0], layer=layer, slot0=2, lse=False)
        assert torch.equal(out, out2)


@pytest.mark.parametrize("K", [1, 6])
def test_q_and_window_inside_a_fused_projection(K):
    B, Hq, Hkv, D = 3, 4, 2, 64
    pool = Pool(10, [18, 0, 140], Hkv=Hkv, D=D)
    qkv = pool.gauss((B, K, (Hq + 2 * Hkv + 1) * D))
    q, k, v = (qkv[..., a * D:b * D].view(B, K, b - a, D) for a, b in ((0, 4), (4, 6), (6, 8)))
    dims = pool.dims(B, K, Hq, q=q, win=k)
    out, lse = attend(pool, B, K, Hq, q, k, v, dims=dims)
    check(pool, B, K, Hq, q, k, v, out, lse)


def test_large_scores_small_scale_and_negative_scale():
    for scale in (4.0, 1e-6, 0.0, -0.3):
        pool = Pool(11, [200, 128, 30], D=64)
        q, k, v = window(pool, 2, 3, 4, q_scale=0.25 if scale == 4.0 else 1.0)
        out, lse = attend(pool, 2, 3, 4, q, k, v, prefix_of=[2, 2], scale=scale)
        check(pool, 2, 3, 4, q, k, v, out, lse, prefix_of=[2, 2], scale=scale)


def test_rising_scores_move_the_running_maximum():
    """Each tile's scores lie far above the tile's before it, and falling ones far below."""
    for sign in (1.0, -1.0):
        pool = Pool(12, [900], D=64, ps=64)
        ramp = torch.linspace(0.0, 3.0, 900, device="cuda")
        for c in range(15):
            n = min(64, 900 - 64 * c)
            pool.k[0, pool.table[0, c], :n] = (ramp[64 * c:64 * c + n, None, None] * sign).to(pool.dtype)
        q = torch.full((1, 2, 4, 64), 0.5, dtype=pool.dtype, device="cuda")
        k, v = pool.gauss((1, 2, 2, 64)), pool.gauss((1, 2, 2, 64))
        out, lse = attend(pool, 1, 2, 4, q, k, v, scale=1.0)
        check(pool, 1, 2, 4, q, k, v, out, lse, scale=1.0)


def test_infinite_values_stay_in_their_window():
    """A value of one sequence's window that is infinite reaches that sequence's rows alone; one in
    pages that a slot no longer covers reaches none."""
    pool = Pool(13, [100, 60, 140], D=64)
    q, k, v = window(pool, 3, 4, 4)
    want, want_lse = attend(pool, 3, 4, 4, q, k, v, prefix_of=[2, 2, -1])
    v2 = v.clone()
    v2[1, 0] = float("inf")
    out, lse = attend(pool, 3, 4, 4, q, k, v2, prefix_of=[2, 2, -1])
    assert torch.equal(lse, want_lse)
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    assert not torch.isfinite(out[1, 0].float()).all()


def torch_reference(pool, B, K, Hq, q, k, v, prefix_of):
    """float64 on the GPU, for sizes beyond the oracle (chains, every window full)."""
    G = Hq // pool.Hkv
    out, lse, mag = [], [], []
    for b in range(B):
        slots = ([prefix_of[b]] if prefix_of is not None and prefix_of[b] >= 0 else []) + [b]
        ks, vs = [], []
        for s in slots:
            n = int(pool.lens[s])
            ids = torch.from_numpy(pool.table[s, :-(-n // pool.ps)]).cuda()
            ks.append(pool.k[0, ids].flatten(0, 1)[:n])
            vs.append(pool.v[0, ids].flatten(0, 1)[:n])
        kk, vv = torch.cat(ks + [k[b]]).double(), torch.cat(vs + [v[b]]).double()
        n = kk.shape[0] - K
        mask = torch.cat([torch.ones(K, n, dtype=torch.bool, device="cuda"),
                          torch.ones(K, K, dtype=torch.bool, device="cuda").tril()], 1)
        x = torch.einsum("thgd,jhd->thgj", q[b].double().view(K, pool.Hkv, G, -1), kk) * pool.D ** -0.5
        x = x.masked_fill(~mask[:, None, None], float("-inf"))
        lse.append(torch.logsumexp(x, -1).view(K, Hq))
        w = torch.softmax(x, -1)
        out.append(torch.einsum("thgj,jhd->thgd", w, vv).reshape(K, Hq, -1))
        mag.append(torch.einsum("thgj,jhd->thgd", w, vv.abs()).reshape(K, Hq, -1))
    return torch.stack(out), torch.stack(lse), torch.stack(mag)


@pytest.mark.parametrize("B,K,Hq,Hkv,D,ps,lens,prefix,dtype", [
    (1, 16, 16, 2, 128, 64, [70001], None, BF),           # one long sequence, split over the card
    (1, 1, 8, 8, 64, 16, [40000], None, HF),
    (24, 16, 16, 2, 128, 128, [1000] * 24 + [5000], 24, BF),
    (100, 1, 24, 4, 128, 16, list(range(100)) + [3001], 100, BF),
    (37, 7, 12, 2, 64, 48, [50 * i for i in range(37)] + [2000], 37, HF),
])
def test_large(B, K, Hq, Hkv, D, ps, lens, prefix, dtype):
    pool = Pool(14, lens, Hkv=Hkv, D=D, ps=ps, dtype=dtype)
    pre = None if prefix is None else [prefix] * B
    q, k, v = window(pool, B, K, Hq)
    out, lse = attend(pool, B, K, Hq, q, k, v, prefix_of=pre)
    ref, ref_lse, mag = torch_reference(pool, B, K, Hq, q, k, v, pre)
    u = ROUND[dtype]
    assert ((out.double() - ref).abs() <= u * (mag + ref.abs()) + 2e-4 * mag).all()
    assert ((lse.double() - ref_lse).abs() <= 1e-4).all()


@pytest.mark.parametrize("B,K,Hq,Hkv,D,plen,own", [
    (60, 1, 8, 4, 64, 20000, 100), (60, 1, 8, 4, 128, 19999, 300), (33, 3, 4, 4, 128, 21000, 500),
    (90, 5, 4, 2, 64, 17000, 260), (7, 16, 6, 6, 128, 15000, 2000), (150, 2, 8, 4, 64, 9000, 129)])
def test_many_tiles_of_both_kinds(B, K, Hq, Hkv, D, plen, own):
    """Enough tiles that prefixes and sequences are dealt out apart: CTAs change from the one to the
    other at any parity, with one or both streams on either side, and several prefixes in turn."""
    lens = [(37 * i) % own for i in range(B)] + [plen, 300]
    pool = Pool(30, lens, Hkv=Hkv, D=D, ps=32)
    pre = [B if i % 20 < 18 else B + 1 if i % 20 == 18 else -1 for i in range(B)]
    q, k, v = window(pool, B, K, Hq)
    out, lse = attend(pool, B, K, Hq, q, k, v, prefix_of=pre)
    ref, ref_lse, mag = torch_reference(pool, B, K, Hq, q, k, v, pre)
    assert ((out.double() - ref).abs() <= ROUND[BF] * (mag + ref.abs()) + 2e-4 * mag).all()
    assert ((lse.double() - ref_lse).abs() <= 1e-4).all()
    again, _ = attend(pool, B, K, Hq, q, k, v, prefix_of=pre)
    assert torch.equal(again, out)


@pytest.mark.parametrize("runs", [1, 3, 700, 1300])
def test_more_sequences_than_the_plan_has_threads(runs):
    """1300 sequences in runs of equal prefixes: fewer and more runs than the plan keeps at hand."""
    B = 1300
    pool = Pool(31, [(7 * i) % 40 for i in range(B)] + [50, 200], Hkv=1, D=64)
    pre = [B + (i * runs // B) % 2 for i in range(B)]
    q, k, v = window(pool, B, 2, 2)
    out, lse = attend(pool, B, 2, 2, q, k, v, prefix_of=pre)
    ref, ref_lse, mag = torch_reference(pool, B, 2, 2, q, k, v, pre)
    assert ((out.double() - ref).abs() <= ROUND[BF] * (mag + ref.abs()) + 2e-4 * mag).all()
    assert ((lse.double() - ref_lse).abs() <= 1e-4).all()


def test_cache_offsets_beyond_32_bits():
    """Pages whose elements lie past 2^32 elements of the pool."""
    ps, Hkv, D = 64, 8, 128
    n_pages = (1 << 32) // (ps * Hkv * D) + 64
    pool = Pool(15, [40, 0], ps=ps, Hkv=Hkv, D=D, n_pages=1, max_pages=4)
    del pool.k, pool.v
    pool.n_pages = n_pages
    pool.k, pool.v = (torch.empty((1, n_pages, ps, Hkv, D), dtype=BF, device="cuda") for _ in range(2))
    pool.table = np.array([[n_pages - 1, n_pages - 20, -1, -1], [n_pages - 7, -1, -1, -1]])
    pool.lens = np.array([100, 33])
    for x in (pool.k, pool.v):
        x[0, n_pages - 25:] = pool.gauss((25, ps, Hkv, D))
    q, k, v = window(pool, 2, 2, 8)
    out, lse = attend(pool, 2, 2, 8, q, k, v, prefix_of=[1, -1])
    ref, ref_lse, mag = torch_reference(pool, 2, 2, 8, q, k, v, [1, -1])
    assert ((out.double() - ref).abs() <= ROUND[BF] * (mag + ref.abs()) + 2e-4 * mag).all()
    assert ((lse.double() - ref_lse).abs() <= 1e-4).all()


def test_runs_repeat_bit_for_bit_and_streams_order():
    """The same call twice on a side stream, its inputs produced just ahead of it and its outputs
    read just behind it."""
    pool = Pool(16, [300, 20, 128, 500], Hkv=2, D=128)
    q, k, v = window(pool, 3, 8, 8)
    want, want_lse = attend(pool, 3, 8, 8, q, k, v, prefix_of=[3, 3, 3])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            q2 = torch.full_like(q, float("nan"))
            torch.mul(q, 1, out=q2)
            out, lse = attend(pool, 3, 8, 8, q2, k, v, prefix_of=[3, 3, 3])
            got = out.clone(), lse.clone()
            out.fill_(0)
    side.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want_lse)


def test_graph_replay():
    """One captured call replayed on new contents and new lengths of its buffers."""
    pool = Pool(17, [300, 20, 128, 500], D=64)
    B, K, Hq = 3, 4, 4
    dims = pool.dims(B, K, Hq)
    q, k, v = window(pool, B, K, Hq)
    table, lens, pre = i32(pool.table), i32(pool.lens), i32([3, 3, -1])
    out, lse = torch.empty_like(q), torch.empty((B, K, Hq), dtype=torch.float32, device="cuda")
    ws = kv.alloc_attn_workspace(dims)
    call = lambda: kv.gdn_attn_verify(dims, 0, q, k, v, pool.k, pool.v, table, lens, pre, None, None,  # noqa: E731
                                      pool.D ** -0.5, out, lse, ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    pool.lens = np.array([130, 5, 128, 17])
    lens.copy_(i32(pool.lens))
    q.copy_(pool.gauss(q.shape))
    out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    check(pool, B, K, Hq, q, k, v, out, lse, prefix_of=[3, 3, -1])


def test_device_status_bits():
    """Lengths, slots, pages, parents and window lengths that only the device can see."""
    gdn.gdn_device_status(clear=True)
    B, K, Hq = 2, 4, 4

    def bits(edit=None, **opt):
        pool = Pool(18, [40, 20, 30], D=64)
        if edit:
            edit(pool)
        q, k, v = window(pool, B, K, Hq)
        out, lse = attend(pool, B, K, Hq, q, k, v, **opt)
        torch.cuda.synchronize()
        return gdn.gdn_device_status(clear=True), out, (pool, q, k, v)

    def set_len(n):
        def f(pool):
            pool.lens = pool.lens.copy()
            pool.lens[0] = n
        return f

    assert bits()[0] == 0
    flags, out, (pool, q, k, v) = bits(set_len(-1))
    assert flags == kv.DEVERR_KV_LEN
    pool.lens[0] = 0  # read as empty
    check(pool, B, K, Hq, q, k, v, out, None)
    assert bits(set_len(1 << 20))[0] == kv.DEVERR_KV_LEN
    flags, out, (pool, q, k, v) = bits(prefix_of=[3, -2])
    assert flags == kv.DEVERR_KV_SLOT
    check(pool, B, K, Hq, q, k, v, out, None)
    flags, out, (pool, q, k, v) = bits(win_len=[9, 4])
    assert flags == kv.DEVERR_KV_WINDOW
    check(pool, B, K, Hq, q, k, v, out, None)
    flags, out, (pool, q, k, v) = bits(parent=[[-1, 0, 2, 2], [-1, 0, 1, 2]])
    assert flags == gdn.DEVERR_TREE_PARENT
    check(pool, B, K, Hq, q, k, v, out, None, parent=[[-1, 0, -1, 2], [-1, 0, 1, 2]])
    for page in (-1, 1 << 27):
        def bad(pool):
            pool.table[0, 0] = page
        flags, out, (pool, q, k, v) = bits(bad)
        assert flags == kv.DEVERR_KV_PAGE
        pool.lens[0], pool.table[0, 0] = 0, 0
        assert torch.isfinite(out[1].float()).all()
