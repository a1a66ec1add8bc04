"""Commit, fork and compact of the paged cache against the oracle: pages move bit for bit, tables,
lengths and reference counts are equal, and no place that a call may not write changes."""
import numpy as np
import pytest
import torch

from kv_util import Pool, i32, random_trees
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


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def books(pool, in_place):
    t = [i32(pool.table), i32(pool.lens), i32(pool.ref)]
    out = t if in_place else [torch.full_like(x, 77) for x in t]
    return t, out


def commit(pool, accept, k, v, parent=None, slot0=0, in_place=True, dims=None, want_bits=0):
    B, K = k.shape[1:3]
    dims = dims or pool.dims(B, K, slot0=slot0)
    ref = O.commit(accept, parent, bits(k), bits(v), bits(pool.k), bits(pool.v), pool.table, pool.lens, pool.ref,
                   pool.ps, slot0)
    t, out = books(pool, in_place)
    kv.gdn_kv_commit(dims, i32(accept), None if parent is None else i32(parent), k, v, pool.k, pool.v,
                     t[0], out[0], t[1], out[1], t[2], out[2], kv.alloc_kv_workspace(dims))
    assert gdn.gdn_device_status(clear=True) == want_bits
    take(pool, out, ref)


def take(pool, out, ref):
    """Compares a call's results with the oracle's, and goes on from them."""
    for got, want in zip([pool.k, pool.v], ref[:2]):
        assert np.array_equal(bits(got), want)
    for got, want in zip(out, ref[2:]):
        assert np.array_equal(got.cpu().numpy(), want)
    pool.table, pool.lens, pool.ref = (x.cpu().numpy().astype(np.int64) for x in out)


def win(pool, B, K):
    return (pool.gauss((pool.layers, B, K, pool.Hkv, pool.D)) for _ in range(2))


@pytest.mark.parametrize("ps,order", [(16, "nhd"), (16, "hnd"), (48, "mixed"), (64, "nhd"), (1024, "hnd")])
@pytest.mark.parametrize("dtype,D,Hkv", [(BF, 128, 3), (HF, 64, 1)])
@pytest.mark.parametrize("tree", [False, True])
def test_commit(ps, order, dtype, D, Hkv, tree):
    B, K = 9, 16
    pool = Pool(1, [0, 1, 15, 16, 17, 31, 32, 40, 63], ps=ps, order=order, dtype=dtype, D=D, Hkv=Hkv, layers=3,
                spare=20, max_pages=12)
    for step in range(3):
        k, v = win(pool, B, K)
        accept = pool.rng.integers(0, K + 1, B)
        commit(pool, accept, k, v, random_trees(pool.rng, B, K) if tree else None, in_place=step != 1)


def test_commit_one_token_and_nothing():
    pool = Pool(2, [16, 5, 0], spare=6)
    for accept in ([1, 1, 1], [0, 0, 0], [0, 1, 0]):
        k, v = win(pool, 3, 1)
        commit(pool, accept, k, v, in_place=False)


def test_commit_whole_prompts_into_later_slots():
    """Windows of many pages (a prefill), into slots 2.. of the table."""
    pool = Pool(3, [7, 0, 0, 3, 16], ps=16, layers=2, spare=60, max_pages=20)
    k, v = win(pool, 3, 200)
    commit(pool, [200, 0, 131], k, v, slot0=2)
    k, v = win(pool, 2, 33)
    commit(pool, [33, 32], k, v)


def test_commit_from_a_fused_projection():
    pool = Pool(4, [3, 30], Hkv=2, D=64, layers=2, spare=8)
    B, K = 2, 5
    kv_all = pool.gauss((2, B, K, 5 * 64))
    k, v = kv_all[..., :128].view(2, B, K, 2, 64), kv_all[..., 192:].view(2, B, K, 2, 64)
    commit(pool, [5, 3], k, v, dims=pool.dims(B, K, win=k))


def test_commit_without_room():
    # two free pages; sequences 0, 2 and 3 need one each, 1 needs none
    pool = Pool(5, [16, 3, 32, 0, 48], spare=2, max_pages=5)
    k, v = win(pool, 5, 4)
    commit(pool, [4, 4, 4, 4, 0], k, v, want_bits=kv.DEVERR_KV_FULL)
    # the table has no further column
    pool = Pool(6, [32, 30], spare=9, max_pages=2)
    k, v = win(pool, 2, 4)
    commit(pool, [1, 2], k, v, want_bits=kv.DEVERR_KV_FULL)
    commit(pool, [0, 1], *win(pool, 2, 4), want_bits=kv.DEVERR_KV_FULL)


def test_commit_refuses_shared_partial_pages_and_bad_lengths():
    pool = Pool(7, [20, 20, 16])
    pool.ref[pool.table[0, 1]] = 2
    commit(pool, [3, 3, 3], *win(pool, 3, 4), want_bits=kv.DEVERR_KV_SHARED)
    commit(pool, [0, 5, -1], *win(pool, 3, 4), want_bits=gdn.DEVERR_ACCEPT_RANGE)


def fork(pool, src, in_place=False, want_bits=0):
    dims = pool.dims()
    ref = O.fork(src, bits(pool.k), bits(pool.v), pool.table, pool.lens, pool.ref, pool.ps)
    t, out = books(pool, False)
    if in_place:
        out[2] = t[2]
    kv.gdn_kv_fork(dims, i32(src), pool.k, pool.v, t[0], out[0], t[1], out[1], t[2], out[2], kv.alloc_kv_workspace(dims))
    assert gdn.gdn_device_status(clear=True) == want_bits
    take(pool, out, ref)


@pytest.mark.parametrize("ps,order", [(16, "nhd"), (32, "hnd"), (48, "mixed"), (1024, "nhd")])
@pytest.mark.parametrize("dtype,D,Hkv", [(BF, 128, 2), (HF, 64, 3)])
def test_fork(ps, order, dtype, D, Hkv):
    n = 12
    pool = Pool(8, [0, 1, 15, 16, 17, 47, 48, 49, 96, 100, 33, 5], ps=ps, order=order, dtype=dtype, D=D, Hkv=Hkv,
                layers=2, spare=60)
    for step in range(4):
        src = pool.rng.integers(-1, n, n)
        fork(pool, src, in_place=step % 2 == 1)


def test_fork_identity_swap_drop_and_one_to_all():
    pool = Pool(9, [20, 33, 0, 16, 7], spare=30)
    for src in ([0, 1, 2, 3, 4], [4, 3, 2, 1, 0], [0, -1, -1, 3, 4], [0, 0, 0, 0, 0], [-1, -1, 2, -1, -1],
                [-1, -1, -1, -1, -1]):
        fork(pool, src)
    assert pool.ref.sum() == 0


def test_fork_without_room_and_with_bad_slots():
    pool = Pool(10, [20, 33, 16], spare=1)
    fork(pool, [0, 0, 0], want_bits=kv.DEVERR_KV_FULL)
    pool = Pool(11, [20, 33, 16], spare=4)
    src = np.array([1, 3, -7])
    dims = pool.dims()
    ref = O.fork([1, -1, -1], bits(pool.k), bits(pool.v), pool.table, pool.lens, pool.ref, pool.ps)
    t, out = books(pool, False)
    kv.gdn_kv_fork(dims, i32(src), pool.k, pool.v, t[0], out[0], t[1], out[1], t[2], out[2], kv.alloc_kv_workspace(dims))
    assert gdn.gdn_device_status(clear=True) == kv.DEVERR_KV_SLOT
    take(pool, out, ref)


def test_forked_sequences_commit_apart():
    """Forks of one sequence share its full pages and write their own next tokens."""
    pool = Pool(12, [37, 0, 0, 0], layers=2, spare=20)
    fork(pool, [0, 0, 0, 0])
    commit(pool, [3, 5, 0, 1], *win(pool, 4, 5))
    assert (pool.ref[pool.table[0, :2]] == 4).all()
    fork(pool, [3, 3, -1, 1], in_place=True)
    commit(pool, [5, 5, 5, 5], *win(pool, 4, 5))


def compact(pool, in_place=True):
    dims = pool.dims()
    k, v, table, ref, live = O.compact(bits(pool.k), bits(pool.v), pool.table, pool.lens, pool.ref, pool.ps)
    t, out = books(pool, in_place)
    n_live = torch.full((1,), -5, dtype=torch.int32, device="cuda")
    kv.gdn_kv_compact(dims, pool.k, pool.v, t[0], out[0], t[1], t[2], out[2], n_live, kv.alloc_kv_workspace(dims))
    assert gdn.gdn_device_status(clear=True) == 0
    assert int(n_live) == live
    take(pool, [out[0], t[1], out[2]], (k, v, table, pool.lens, ref))
    assert (pool.ref[:live] > 0).all() and (pool.ref[live:] == 0).all()


@pytest.mark.parametrize("ps,order", [(16, "nhd"), (16, "hnd"), (48, "mixed")])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype,D,Hkv", [(BF, 128, 2), (HF, 64, 3)])
def test_compact(ps, order, in_place, dtype, D, Hkv):
    pool = Pool(13, [0, 1, 100, 16, 250, 47, 300], ps=ps, order=order, dtype=dtype, D=D, Hkv=Hkv, layers=2, spare=40)
    compact(pool, in_place)
    compact(pool, in_place)                    # nothing left to move
    fork(pool, [2, 2, -1, -1, 4, -1, 0])       # shared pages, and holes
    compact(pool, in_place)


def test_compact_nothing_live_everything_live_one_page():
    compact(Pool(14, [0, 0], spare=7))
    compact(Pool(15, [64, 31], spare=0))
    compact(Pool(16, [1], spare=0))
    compact(Pool(17, [0], spare=1))


@pytest.mark.parametrize("n_pages", [1023, 1024, 1025, 5000, 70001])
def test_plans_over_many_pages(n_pages):
    """Pools around and beyond what the plan's threads take in one step; the free pages lie late."""
    rng = np.random.default_rng(n_pages)
    pool = Pool(18, [16 * 7, 5, 40], Hkv=1, n_pages=n_pages, max_pages=2000)
    pool.ref[pool.ref == 0] = 3                # held by others
    late = rng.choice(np.flatnonzero(pool.ref == 3), 9, replace=False)
    pool.ref[late] = 0
    commit(pool, [16, 3, 9], *win(pool, 3, 16), in_place=False)
    fork(pool, [0, 1, 1])
    compact(pool)


def test_many_slots():
    """More slots than the plan has threads."""
    n = 1500
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 40, n)
    pool = Pool(19, lens, Hkv=1, spare=3000, max_pages=4)
    fork(pool, rng.integers(-1, n, n))
    commit(pool, rng.integers(0, 5, n), *win(pool, n, 4), in_place=False)
    compact(pool)


def test_offsets_beyond_32_bits():
    ps, Hkv, D = 64, 8, 128
    n_pages = (1 << 32) // (ps * Hkv * D) + 64
    dims = kv.make_kv_dims(2, 4, Hkv, Hkv, D, ps, n_pages, 4)
    k, v = (torch.zeros((1, n_pages, ps, Hkv, D), dtype=BF, device="cuda") for _ in range(2))
    top = n_pages - 1
    ref = np.ones(n_pages)
    ref[[n_pages - 3, n_pages - 2]] = 0
    k[0, top], v[0, top] = 1.0, 2.0
    table, lens = i32([[top, -1, -1, -1], [5, -1, -1, -1]]), i32([62, 64])
    kw, vw = (torch.full((1, 2, 4, Hkv, D), x, dtype=BF, device="cuda") for x in (3.0, 4.0))
    ws, r = kv.alloc_kv_workspace(dims), i32(ref)
    kv.gdn_kv_commit(dims, i32([4, 4]), None, kw, vw, k, v, table, table, lens, lens, r, r, ws)
    assert table.cpu().tolist() == [[top, n_pages - 3, -1, -1], [5, n_pages - 2, -1, -1]]
    assert (k[0, top, 62:] == 3).all() and (k[0, top, :62] == 1).all() and (v[0, n_pages - 3, :2] == 4).all()
    assert (v[0, n_pages - 2, :4] == 4).all() and (v[0, n_pages - 2, 4:] == 0).all()
    t2, l2 = torch.empty_like(table), torch.empty_like(lens)
    r[7] = 0
    kv.gdn_kv_fork(dims, i32([0, 0]), k, v, table, t2, lens, l2, r, r, ws)
    assert t2.cpu().tolist() == [[top, n_pages - 3, -1, -1], [top, 7, -1, -1]] and l2.cpu().tolist() == [66, 66]
    assert (k[0, 7, :2] == 3).all() and (k[0, 7, 2:] == 0).all()


def test_graph_replay_of_commit_in_place():
    pool = Pool(20, [10, 16, 3], layers=2, spare=30, max_pages=6)
    k, v = win(pool, 3, 4)
    dims = pool.dims(3, 4)
    t, _ = books(pool, True)
    acc, ws = i32([2, 4, 1]), kv.alloc_kv_workspace(dims)
    call = lambda: kv.gdn_kv_commit(dims, acc, None, k, v, pool.k, pool.v, t[0], t[0], t[1], t[1], t[2], t[2], ws)  # noqa: E731
    none = i32([0, 0, 0])
    kv.gdn_kv_commit(dims, none, None, k, v, pool.k, pool.v, t[0], t[0], t[1], t[1], t[2], t[2], ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(4):
        accept = pool.rng.integers(0, 5, 3)
        acc.copy_(i32(accept))
        for x in (k, v):
            x.copy_(pool.gauss(x.shape))
        ref = O.commit(accept, None, bits(k), bits(v), bits(pool.k), bits(pool.v), pool.table, pool.lens, pool.ref, pool.ps)
        graph.replay()
        take(pool, t, ref)
