"""Host side of the paged cache's C ABI, and pins of its oracle.

Every library call here is built to fail validation, which happens before the library touches
CUDA: no GPU is needed and no kernel is launched."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

from oracle import kv_oracle as O
from speculative_decode_verify_gdn_gb300 import build, gdn, kv

torch = pytest.importorskip("torch")
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gdn_kv.h")


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return kv.load_library()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?\w+\s*\**\s*(gdn_\w+)\s*\(", text, flags=re.M))
    assert names == set(kv.EXPORTED)
    for n in names:
        assert hasattr(lib, n), n


def test_status_bits_are_those_of_the_header():
    text = open(HEADER).read()
    for name in ("LEN", "PAGE", "SLOT", "FULL", "SHARED", "WINDOW"):
        assert int(re.search(rf"GDN_DEVERR_KV_{name} (\d+)u", text).group(1)) == getattr(kv, f"DEVERR_KV_{name}")


def test_the_digest_of_the_build_covers_the_header(tmp_path, monkeypatch):
    before = build._digest(), build.kernel_source_digest(), build.verify_kernel_digest()
    other = tmp_path / "gdn_kv.h"
    other.write_text(open(HEADER).read() + "\nint more;\n")
    monkeypatch.setattr(build, "KV_HEADER", str(other))
    after = build._digest(), build.kernel_source_digest(), build.verify_kernel_digest()
    assert before[0] != after[0] and before[1] != after[1] and before[2] == after[2]


BASE = dict(B=2, K=4, Hq=4, Hkv=2, D=64, page_size=16, n_pages=10, max_pages=4, n_slots=3, n_layers=2)
P, MB = 1 << 32, 1 << 24     # never dereferenced
BIG = ctypes.c_uint64(1 << 40)


def ptrs(n):
    return [P + i * MB for i in range(n)]


def dims(**over):
    return kv.make_kv_dims(**dict(BASE, **over))


def with_field(name, value, **over):
    d = dims(**over)
    setattr(d, name, value)
    return d


def attn(lib, d, args=None, layer=0, scale=0.125, ws=BIG, last=None):
    a = ptrs(13) if args is None else args
    # q k_win v_win k_cache v_cache table seq_len prefix_of win_len parent | out lse workspace
    return lib.gdn_attn_verify(None if d is None else ctypes.byref(d), layer, *a[:10], scale, *a[10:13], ws, None)


def commit(lib, d, args=None, ws=BIG):
    a = ptrs(13) if args is None else args
    return lib.gdn_kv_commit(None if d is None else ctypes.byref(d), *a, ws, None)


def fork(lib, d, args=None, ws=BIG):
    return lib.gdn_kv_fork(None if d is None else ctypes.byref(d), *(ptrs(10) if args is None else args), ws, None)


def compact(lib, d, args=None, ws=BIG):
    return lib.gdn_kv_compact(None if d is None else ctypes.byref(d), *(ptrs(9) if args is None else args), ws, None)


INV, UNS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("name,value,status", [
    ("Hkv", 0, INV), ("D", 96, UNS), ("D", 256, UNS), ("page_size", 8, UNS), ("page_size", 24, UNS),
    ("page_size", 2048, UNS), ("n_pages", 0, INV), ("n_pages", (1 << 28) + 1, INV), ("n_slots", 0, INV),
    ("max_pages", 0, INV), ("max_pages", 1 << 30, INV), ("n_layers", 0, INV), ("dtype", 2, INV),
    ("cache_token_stride", 60, INV), ("cache_token_stride", 132, INV), ("cache_head_stride", 8, INV),
    ("cache_page_stride", 64, INV), ("cache_layer_stride", 128, INV), ("cache_page_stride", 1 << 40, INV)])
def test_cache_dims_are_checked_by_every_call(lib, name, value, status):
    d = with_field(name, value)
    for call in (attn, commit, fork, compact):
        assert call(lib, d) == status, call
        assert gdn.last_error() != ""


@pytest.mark.parametrize("name,value,status", [
    ("B", -1, INV), ("B", 65536, INV), ("slot0", -1, INV), ("slot0", 2, INV), ("K", 0, UNS), ("K", 17, UNS),
    ("Hq", 0, INV), ("Hq", 5, UNS), ("q_token_stride", 200, INV), ("q_token_stride", 258, INV),
    ("win_token_stride", 64, INV), ("win_token_stride", 130, INV)])
def test_attention_dims(lib, name, value, status):
    assert attn(lib, with_field(name, value)) == status
    assert gdn.last_error() != ""
    n = ctypes.c_uint64(0)
    d = with_field(name, value)
    assert lib.gdn_attn_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status


def test_attention_arguments(lib):
    d = dims()
    assert attn(lib, None) == INV and "dims" in gdn.last_error()
    assert attn(lib, d, layer=2) == INV and attn(lib, d, layer=-1) == INV and "layer" in gdn.last_error()
    assert attn(lib, d, scale=float("nan")) == INV and attn(lib, d, scale=float("inf")) == INV
    assert attn(lib, d, ws=ctypes.c_uint64(16)) == INV and "workspace" in gdn.last_error()
    for i in range(13):
        if i not in (7, 8, 9, 11):
            a = ptrs(13)
            a[i] = None
            assert attn(lib, d, a) == INV and "NULL" in gdn.last_error(), i
        a = ptrs(13)
        a[i] += 2
        assert attn(lib, d, a) == INV and "aligned" in gdn.last_error(), i
    for i in range(10):          # an output over an input
        for o in (10, 11, 12):
            a = ptrs(13)
            a[o] = a[i]
            assert attn(lib, d, a) == gdn.GDN_ERR_ALIAS, (i, o)
    a = ptrs(13)
    a[11] = a[10]
    assert attn(lib, d, a) == gdn.GDN_ERR_ALIAS
    assert attn(lib, dims(B=0), [None] * 13) == gdn.GDN_OK
    assert gdn.last_error() == ""


@pytest.mark.parametrize("name,value,status", [("B", -1, INV), ("slot0", 2, INV), ("K", 0, UNS), ("K", 17, UNS),
                                               ("win_token_stride", 64, INV), ("win_layer_stride", 12, INV)])
def test_commit_dims(lib, name, value, status):
    assert commit(lib, with_field(name, value)) == status   # (K = 17: a tree; a chain may be longer)
    assert gdn.last_error() != ""


@pytest.mark.parametrize("call,n,inputs,outputs,optional,in_place", [
    (commit, 13, (0, 1, 2, 3, 6, 8, 10), (4, 5, 7, 9, 11, 12), (1,), {(7, 6), (9, 8), (11, 10)}),
    (fork, 10, (0, 3, 5, 7), (1, 2, 4, 6, 8, 9), (), {(8, 7)}),
    (compact, 9, (2, 4, 5), (0, 1, 3, 6, 7, 8), (), {(3, 2), (6, 5)})])
def test_pool_arguments(lib, call, n, inputs, outputs, optional, in_place):
    d = dims()
    assert call(lib, None) == INV
    assert call(lib, d, ws=ctypes.c_uint64(16)) == INV and "workspace" in gdn.last_error()
    for i in range(n):
        if i not in optional:
            a = ptrs(n)
            a[i] = None
            assert call(lib, d, a) == INV and "NULL" in gdn.last_error(), i
        a = ptrs(n)
        a[i] += 2
        assert call(lib, d, a) == INV and "aligned" in gdn.last_error(), i
    for o in outputs:
        for i in inputs:
            if (o, i) not in in_place:
                a = ptrs(n)
                a[o] = a[i]
                assert call(lib, d, a) == gdn.GDN_ERR_ALIAS, (o, i)
    for o, i in in_place:        # shifted by one entry is not in place
        a = ptrs(n)
        a[o] = a[i] + 4
        assert call(lib, d, a) == gdn.GDN_ERR_ALIAS, (o, i)
    for x, o in enumerate(outputs):
        for o2 in outputs[x + 1:]:
            a = ptrs(n)
            a[o2] = a[o]
            assert call(lib, d, a) == gdn.GDN_ERR_ALIAS, (o, o2)


def test_workspace_sizes(lib):
    small, large = dims(), dims(B=3, n_slots=4, n_pages=20)
    assert 0 < kv.gdn_kv_workspace_size(small) <= kv.gdn_kv_workspace_size(large)
    assert 0 < kv.gdn_attn_workspace_size(small) <= kv.gdn_attn_workspace_size(large)
    with pytest.raises(gdn.GdnError):
        kv.gdn_kv_workspace_size(with_field("D", 80))
    assert lib.gdn_kv_workspace_size(ctypes.byref(small), None) == INV


def test_dims_take_strides_from_views():
    k = torch.empty(2, 10, 2, 16, 64).transpose(2, 3)        # [layers, pages, heads, tokens, D] in memory
    d = kv.make_kv_dims(**BASE, cache=k)
    assert (d.cache_token_stride, d.cache_head_stride, d.cache_page_stride) == (64, 1024, 2048)
    qkv = torch.empty(2, 4, 9 * 64)
    q, w = qkv[..., :256].view(2, 4, 4, 64), qkv[..., 256:384].view(2, 4, 2, 64)
    d = kv.make_kv_dims(**BASE, q=q, win=w)
    assert d.q_token_stride == 576 and d.win_token_stride == 576
    with pytest.raises(ValueError):
        kv.make_kv_dims(**dict(BASE, dtype=torch.float32))


def test_binding_refuses_cpu_tensors_and_wrong_types():
    d = dims()
    t = torch.zeros(4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kv.gdn_attn_verify(d, 0, t, t, t, t, t, t, t, None, None, None, 1.0, t, None, t)
    with pytest.raises(TypeError):
        kv.gdn_kv_fork(d, None, None, None, t, t, t, t, t, t, t)


# ---------------------------------------------------------------- the oracle
def test_attention_oracle_against_matrix_softmax_and_by_hand():
    # two equal keys share the weight; a third at score log 2 more gets half of all
    q = np.array([[[[1.0, 0.0]]]])
    k = np.array([[[0.0, 5.0]], [[0.0, -1.0]], [[math.log(2.0), 0.0]]])
    v = np.array([[[1.0, 0.0]], [[3.0, 0.0]], [[0.0, 8.0]]])
    cache_k, cache_v = k[:2].reshape(1, 2, 1, 2), v[:2].reshape(1, 2, 1, 2)
    out, lse = O.attention(q, k[2:].reshape(1, 1, 1, 2), v[2:].reshape(1, 1, 1, 2), cache_k, cache_v, [[0]], [2], None,
                           None, None, 1.0)
    assert np.allclose(out[0, 0, 0], [1.0, 4.0]) and np.allclose(lse, math.log(4.0))
    rng = np.random.default_rng(0)
    B, K, Hq, Hkv, D, ps = 2, 3, 4, 2, 8, 4
    ck, cv = rng.normal(size=(2, 9, ps, Hkv, D))
    table, lens = np.array([[8, 1, -1], [3, 4, 6], [0, 7, -1]]), np.array([5, 11, 8])
    q, kw, vw = rng.normal(size=(B, K, Hq, D)), rng.normal(size=(B, K, Hkv, D)), rng.normal(size=(B, K, Hkv, D))
    out, lse = O.attention(q, kw, vw, ck, cv, table, lens, [2, -1], None, None, 0.3)
    for b in range(B):
        rows = ([0, 7] if b == 0 else []) + [p for p in table[b] if p >= 0]
        n = (8 if b == 0 else 0) + lens[b]
        kk = np.concatenate([ck[rows].reshape(-1, Hkv, D)[:n], kw[b]])
        vv = np.concatenate([cv[rows].reshape(-1, Hkv, D)[:n], vw[b]])
        mask = np.concatenate([np.ones((K, n)), np.tril(np.ones((K, K)))], 1) > 0
        for h in range(Hq):
            x = np.where(mask, 0.3 * q[b, :, h] @ kk[:, h // 2].T, -np.inf)
            w = np.exp(x) / np.exp(x).sum(1, keepdims=True)
            assert np.allclose(out[b, :, h], w @ vv[:, h // 2])
            assert np.allclose(lse[b, :, h], np.log(np.exp(x).sum(1)))


def test_attention_oracle_splits_its_keys_anywhere():
    """A prefix and an own part give what one sequence of both gives; a tree row what its path's chain gives."""
    rng = np.random.default_rng(1)
    ck, cv = rng.normal(size=(2, 6, 4, 1, 8))
    q, kw, vw = (rng.normal(size=(1, 4, 1, 8)) for _ in range(3))
    table = np.array([[0, 1], [2, 3]])
    joined = np.array([[2, 3, 0, 1]])
    a = O.attention(q, kw, vw, ck, cv, table, [6, 8], [1], None, None, 1.0)
    b = O.attention(q, kw, vw, ck, cv, joined, [14], None, None, None, 1.0)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])
    parent = [[-1, 0, 0, 1]]
    tree = O.attention(q, kw, vw, ck, cv, table, [6, 8], None, None, parent, 1.0)
    path = [0, 1, 3]
    chain = O.attention(q[:, path], kw[:, path], vw[:, path], ck, cv, table, [6, 8], None, None, None, 1.0)
    assert np.allclose(tree[0][:, path], chain[0]) and np.allclose(tree[1][:, path], chain[1])
    # padding rows are empty
    out, lse = O.attention(q, kw, vw, ck, cv, table, [6, 8], [1], [2], None, 1.0)
    assert (out[:, 2:] == 0).all() and np.isneginf(lse[:, 2:]).all()


def test_commit_oracle_by_hand():
    ck = np.zeros((1, 4, 2, 1, 1))
    kw = np.arange(1, 5, dtype=float).reshape(1, 1, 4, 1, 1)
    table, lens, ref = np.array([[2, -1, -1]]), np.array([1]), np.array([0, 7, 1, 0])
    k, v, t, n, r = O.commit([3], None, kw, -kw, ck, ck, table, lens, ref, 2)
    assert t.tolist() == [[2, 0, -1]] and n.tolist() == [4] and r.tolist() == [1, 7, 1, 0]
    assert k[0, 2, :, 0, 0].tolist() == [0, 1] and k[0, 0, :, 0, 0].tolist() == [2, 3] and (v == -k).all()
    # the path to node 3 of a tree
    k, _, _, n, _ = O.commit([4], [[-1, 0, 0, 2]], kw, kw, ck, ck, table, lens, ref, 2)
    assert n.tolist() == [4] and k[0, 0, :, 0, 0].tolist() == [3, 4] and k[0, 2, 1, 0, 0] == 1


def test_fork_and_compact_oracles_keep_every_sequence():
    rng = np.random.default_rng(2)
    ps, n = 4, 6
    lens = np.array([0, 3, 4, 9, 16, 6])
    pages = -(-lens // ps)
    ids = rng.permutation(40)
    table, ref, at = np.full((n, 5), -1), np.zeros(40, dtype=int), 0
    for s in range(n):
        table[s, :pages[s]] = ids[at:at + pages[s]]
        ref[table[s, :pages[s]]] = 1
        at += pages[s]
    ck, cv = rng.normal(size=(2, 2, 40, ps, 1, 3))

    def tokens(k, t, ln):
        return [[O.gather(k[layer], t[s], ln[s]) for layer in range(2)] for s in range(n)]

    def count(t, ln):
        r = np.zeros(40, dtype=int)
        for s in range(n):
            np.add.at(r, t[s, :-(-ln[s] // ps)], 1)
        return r

    before = tokens(ck, table, lens)
    src = [3, 3, -1, 5, 3, 2]
    k, v, t, ln, r = O.fork(src, ck, cv, table, lens, ref, ps)
    after = tokens(k, t, ln)
    for i, s in enumerate(src):
        want = before[s] if s >= 0 else [np.zeros((0, 1, 3))] * 2
        assert all(np.array_equal(a, b) for a, b in zip(after[i], want))
    assert np.array_equal(r, count(t, ln))
    k2, v2, t2, r2, live = O.compact(k, v, t, ln, r, ps)
    assert live == (r > 0).sum() and (r2[:live] > 0).all() and (r2[live:] == 0).all()
    assert np.array_equal(r2, count(t2, ln))
    for a, b in zip(tokens(k2, t2, ln), after):
        assert all(np.array_equal(x, y) for x, y in zip(a, b))
