"""Attention over the paged cache at its limits.  Tolerances are those of test_gpu_kv_attn.py."""
import numpy as np
import pytest
import torch

from kv_util import ROUND, Pool, i32, random_trees
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


@pytest.mark.parametrize("ps", [16, 48, 112])
def test_the_longest_slot(ps):
    """A slot of nearly 2^30 tokens whose columns name one page of negligible weight, but for a few
    marked ones beyond 2^29 tokens and the last: each of their tokens has its share of the output."""
    rng = np.random.default_rng(ps)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(ps)
    D, cols = 64, (1 << 30) // ps
    n = cols * ps - 7
    marks = np.unique(np.concatenate([rng.integers((1 << 29) // ps, cols, 60), [(1 << 29) // ps + 2, 939524192 // ps,
                                                                                 cols - 2, cols - 1]]))
    pages = 1 + len(marks)
    k, v = (torch.empty((1, pages, ps, 1, D), dtype=BF, device="cuda").normal_(generator=gen) for _ in range(2))
    k[0, 0, :, 0, 0] = -64.0          # e^-64 of 2^30 tokens: 2e-19 of the sum
    table = torch.zeros((1, cols), dtype=torch.int32, device="cuda")
    table[0, torch.from_numpy(marks).cuda()] = torch.arange(1, pages, dtype=torch.int32, device="cuda")
    k[0, -1, ps - 7:], v[0, -1, ps - 7:] = float("nan"), float("nan")
    q = torch.zeros((1, 1, 1, D), dtype=BF, device="cuda")
    q[..., 0] = 1.0
    kw, vw = (torch.empty((1, 1, 1, D), dtype=BF, device="cuda").normal_(generator=gen) for _ in range(2))
    out, lse = torch.empty_like(q), torch.empty((1, 1, 1), dtype=torch.float32, device="cuda")
    dims = kv.make_kv_dims(1, 1, 1, 1, D, ps, pages, cols)
    kv.gdn_attn_verify(dims, 0, q, kw, vw, k, v, table, i32([n]), None, None, None, 1.0, out, lse, kv.alloc_attn_workspace(dims))
    keys = torch.cat([k[0, 1:].reshape(-1, D)[:-7], kw.view(1, D)]).double()
    values = torch.cat([v[0, 1:].reshape(-1, D)[:-7], vw.view(1, D)]).double()
    w = torch.softmax(keys[:, 0], 0)
    ref, mag = w @ values, w @ values.abs()
    assert ((out.view(D).double() - ref).abs() <= ROUND[BF] * (mag + ref.abs()) + 2e-4 * mag).all()
    assert abs(lse.item() - torch.logsumexp(keys[:, 0], 0).item()) <= 1e-4


def test_parents_of_padding_tokens_are_not_read():
    """Whatever a tree holds behind a window's tokens, no status bit is set and no row changes."""
    B, K, Hq = 5, 9, 4
    pool = Pool(40, [20, 0, 130, 7, 64])
    win = np.array([0, 1, 4, 8, 9])
    par = random_trees(pool.rng, B, K)
    q, k, v = (pool.gauss((B, K, h, pool.D)) for h in (Hq, pool.Hkv, pool.Hkv))
    dims = pool.dims(B, K, Hq)
    ws, results = kv.alloc_attn_workspace(dims), []
    for fill in (None, 99, -7, K - 1, -(1 << 31), (1 << 31) - 1):
        p = par.copy()
        if fill is not None:
            p[np.arange(K)[None, :] >= win[:, None]] = fill
        out, lse = torch.empty_like(q), torch.empty((B, K, Hq), dtype=torch.float32, device="cuda")
        kv.gdn_attn_verify(dims, 0, q, k, v, pool.k, pool.v, i32(pool.table), i32(pool.lens), None, i32(win), i32(p),
                           pool.D ** -0.5, out, lse, ws)
        assert gdn.gdn_device_status(clear=True) == 0, fill
        results.append((out, lse))
    assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(r, results[0]))


def test_segments_of_many_seconds():
    """More sequences of 3 x 2^28 tokens, a pair of row tiles each, than there are CTAs: each works on a
    segment for ten seconds with another behind it, and no bounded wait takes that for a fault.  The
    columns name pages of negligible weight but for one."""
    D, ps, B, K, G = 64, 1024, 153, 16, 16
    cols = 3 * (1 << 28) // ps
    n = cols * ps - 5
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    k, v = (torch.empty((1, 65, ps, 1, D), dtype=BF, device="cuda").normal_(generator=gen) for _ in range(2))
    k[0, :64, :, 0, 0] = -64.0
    table = (torch.arange(cols, dtype=torch.int32, device="cuda") % 64).repeat(B, 1)
    table[:, cols - 2] = 64
    q = torch.zeros((B, K, G, D), dtype=BF, device="cuda")
    q[..., 0] = 1.0
    kw, vw = (torch.empty((B, K, 1, D), dtype=BF, device="cuda").normal_(generator=gen) for _ in range(2))
    out, lse = torch.empty_like(q), torch.empty((B, K, G), dtype=torch.float32, device="cuda")
    dims = kv.make_kv_dims(B, K, G, 1, D, ps, 65, cols)
    kv.gdn_attn_verify(dims, 0, q, kw, vw, k, v, table, i32([n] * B), None, None, None, 1.0, out, lse,
                       kv.alloc_attn_workspace(dims))
    torch.cuda.synchronize()
    assert gdn.gdn_device_status(clear=True) == 0
    keys = torch.cat([k[0, 64, :, 0].expand(B, ps, D), kw[:, :, 0]], 1).double()
    values = torch.cat([v[0, 64, :, 0].expand(B, ps, D), vw[:, :, 0]], 1).double()
    seen = torch.cat([torch.ones(K, ps, device="cuda"), torch.ones(K, K, device="cuda").tril()], 1) > 0
    scores = keys[:, None, :, 0].expand(B, K, -1).masked_fill(~seen, float("-inf"))
    w = torch.softmax(scores, 2)
    ref, mag = (w @ values)[:, :, None], (w @ values.abs())[:, :, None]
    assert ((out.double() - ref).abs() <= ROUND[BF] * (mag + ref.abs()) + 2e-4 * mag).all()
    assert ((lse.double() - torch.logsumexp(scores, 2)[:, :, None]).abs() <= 1e-4).all()


@pytest.mark.parametrize("page", [-1, 1 << 27])
@pytest.mark.parametrize("shared", [False, True])
def test_a_bad_page_leaves_the_other_sequences_alone(page, shared):
    """A page number outside the pool in one sequence's row (or in the prefix of two): the sequences that
    do not read it get the results that they get without it."""
    B, K, Hq = 5, 3, 4
    pre = [5, 5, 6, 6, -1]
    pool = Pool(41, [40, 300, 17, 0, 130, 90, 200], D=64)
    q, k, v = (pool.gauss((B, K, h, pool.D)) for h in (Hq, pool.Hkv, pool.Hkv))
    dims = pool.dims(B, K, Hq)
    ws, results = kv.alloc_attn_workspace(dims), []
    for bad in (False, True):
        table = pool.table.copy()
        if bad:
            table[5 if shared else 1, 0] = page
        out, lse = torch.empty_like(q), torch.empty((B, K, Hq), dtype=torch.float32, device="cuda")
        kv.gdn_attn_verify(dims, 0, q, k, v, pool.k, pool.v, i32(table), i32(pool.lens), i32(pre), None, None,
                           pool.D ** -0.5, out, lse, ws)
        assert gdn.gdn_device_status(clear=True) == (kv.DEVERR_KV_PAGE if bad else 0)
        results.append((out, lse))
    for b in [2, 3, 4] + ([] if shared else [0]):
        assert all(torch.equal(x[b], y[b]) for x, y in zip(*results)), b
