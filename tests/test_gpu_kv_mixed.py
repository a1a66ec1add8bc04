"""Prefill attention of batches that hold single tokens and chunks of prompts side by side: the kernels for few rows and
for tiles each take their sequences.  Tolerances are those of test_gpu_kv_prefill.py, whose helpers these tests use."""
import numpy as np
import pytest
import torch

from kv_util import Pool, i32
from speculative_decode_verify_gdn_gb300 import gdn, kv
from speculative_decode_verify_gdn_gb300.build import build_library
from test_gpu_kv_prefill import attend, run_case

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


def batch(B, G, rng):
    """Tokens and lengths of B sequences, on average at most 8 rows of G heads: single tokens, none, a few around the
    8 rows, and chunks at the first, a middle and the last sequence."""
    few = 8 // G
    new = np.where(rng.random(B) < 0.25, 0, 1)
    new[[3, 8, B - 4]] = few, few + 1, 2 * few
    chunks = rng.permutation([17, 40, 1 + few])
    for b, n in zip((0, B // 2, B - 1), chunks):
        new[b] = n
    lens = new + rng.integers(0, 200, B)
    lens[[1, 2]] = new[[1, 2]]
    lens[5], lens[B // 2] = 0, max(1, int(new[B // 2]) - 9)     # rows without keys, in a chunk and alone
    return new, lens


# max_pages is that of a table for long slots: what few rows would read at worst is then too much to let them take all
@pytest.mark.parametrize("G", [1, 2, 3, 4])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,dtype,ps", [(64, HF, 16), (128, BF, 64)])
@pytest.mark.parametrize("wide_table", [False, True])
def test_chunks_among_single_tokens(G, causal, D, dtype, ps, wide_table):
    rng = np.random.default_rng(10 * G + D)
    B = 70
    new, lens = batch(B, G, rng)
    assert 32 <= new.sum() != B and new.sum() * G <= 8 * B
    pre = np.where(rng.random(B) < 0.5, B, -1)
    pool, cu, q, out, lse = run_case(90 + G, new, lens, 2 * G, causal, prefixes=[150], pre=pre, D=D, dtype=dtype, ps=ps, spare_rows=2,
                                     max_pages=1 << 16 if wide_table else None)
    again = attend(pool, cu, q, causal, pre=pre)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("wide_table", [False, True])
@pytest.mark.parametrize("spare", [0, 3])
@pytest.mark.parametrize("B", [5, 40, 300])
def test_as_many_tokens_as_sequences_all_of_one(B, spare, wide_table):
    """B tokens of one sequence among B, whose keys are fewer, as many or more."""
    for which, n_keys in ((0, B - 2), (B // 2, B), (B - 1, B + 700)):
        new, lens = np.zeros(B, dtype=int), np.full(B, 9)
        new[which], lens[which] = B, n_keys
        run_case(95, new, lens, 4, True, Hkv=2, D=128, ps=32, spare_rows=spare, max_pages=1 << 16 if wide_table else None)


def test_long_axes_of_both_kinds():
    """A chunk and single tokens behind thousands of keys: both kernels' items are cut into pieces, which share a
    workspace."""
    for D, Hkv in ((128, 2), (64, 4)):
        new = [1] * 40 + [60, 0, 5]
        lens = [3000, 10, 700, 5000] * 10 + [9000, 20, 4000]
        pool, cu, q, out, lse = run_case(96, new, lens, 2 * Hkv, True, Hkv=Hkv, D=D, ps=64, max_pages=1 << 16)
        for _ in range(3):
            again = attend(pool, cu, q, True)
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_what_is_wrong_with_one_kind_leaves_the_other_alone():
    pool = Pool(97, [50] * 39 + [200], D=64, ps=16, max_pages=1 << 16)
    cu = np.concatenate([[0], np.cumsum([1] * 39 + [30])])
    q = pool.gauss((int(cu[-1]), 4, 64), 2.0)
    want = attend(pool, cu, q, True)
    for slot, column, others in ((39, 3, slice(0, 39)), (7, 1, [*range(7), *range(8, 69)])):
        table = pool.table.copy()
        table[slot, column] = 1 << 27
        got = attend(pool, cu, q, True, table=table)
        assert gdn.gdn_device_status(clear=True) == kv.DEVERR_KV_PAGE
        assert all(torch.equal(a[others], b[others]) for a, b in zip(want, got))
        lens = pool.lens.copy()
        lens[slot] = -3
        got = attend(pool, cu, q, True, lens=lens)
        assert gdn.gdn_device_status(clear=True) == kv.DEVERR_KV_LEN
        assert all(torch.equal(a[others], b[others]) for a, b in zip(want, got))
        rows = slice(int(cu[slot]), int(cu[slot + 1]))
        assert (got[0][rows] == 0).all() and torch.isneginf(got[1][rows]).all()
    bad = cu.copy()
    bad[5] = 70
    got = attend(pool, bad, q, True)
    assert gdn.gdn_device_status(clear=True) == gdn.DEVERR_SEQLENS
    assert (got[0] == 9.0).all() and (got[1] == 9.0).all()


def test_a_chunk_does_not_wait_for_few_rows():
    """255 single tokens and a chunk of 257 behind 65536 in one call take at most four times what a call for each kind
    takes (a few rows at a time through the chunk's keys: more than eight times)."""
    B, Hq, Hkv, D, ps = 256, 32, 8, 128, 64
    lens = [500] * 255 + [65536]
    pages = [-(-n // ps) for n in lens]
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    ids = torch.randperm(sum(pages)).int()
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = ids[at:at + n]
        at += n
    table, held = table.cuda(), i32(lens)
    k, v = (torch.empty((1, sum(pages), ps, Hkv, D), dtype=BF, device="cuda").normal_() for _ in range(2))

    def call(new, slot0):
        cu = i32(np.concatenate([[0], np.cumsum(new)]))
        q = torch.empty((sum(new), Hq, D), dtype=BF, device="cuda").normal_()
        d = kv.make_kv_dims(len(new), 1, Hq, Hkv, D, ps, sum(pages), max(pages), B, slot0)
        out, ws = torch.empty_like(q), kv.alloc_attn_prefill_workspace(d, sum(new))
        return lambda: kv.gdn_attn_prefill(d, 0, cu, q, k, v, table, held, None, True, D ** -0.5, out, None, ws)

    def best(f):
        times = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            a.record()
            f()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times[3:])

    single, chunk, both = best(call([1] * 255, 0)), best(call([257], 255)), best(call([1] * 255 + [257], 0))
    assert both <= 4 * (single + chunk), (single, chunk, both)
