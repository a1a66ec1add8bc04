"""Attention of packed queries over the paged cache against the float64 oracle.  Tolerances are those of
test_gpu_kv_attn.py: |out - ref| <= u (A + |ref|) + 2e-4 A with A = sum_j w_j |v_j|, and |lse - ref| <= 1e-4."""
import numpy as np
import pytest
import torch

from kv_util import ROUND, Pool, f64, i32
from oracle import prompt_oracle as O
from speculative_decode_verify_gdn_gb300 import gdn, kv
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


def attend(pool, cu, q, causal, pre=None, layer=0, slot0=0, scale=None, lse=True, dims=None, table=None, lens=None):
    B = len(cu) - 1
    N, Hq, D = q.shape
    d = dims or kv.make_kv_dims(B, 1, Hq, pool.Hkv, D, pool.ps, pool.n_pages, pool.max_pages, len(pool.lens), slot0, pool.layers,
                                pool.dtype, cache=pool.k, q=q)
    out = torch.full((N, Hq, D), 9.0, dtype=pool.dtype, device="cuda")
    ls = torch.full((N, Hq), 9.0, dtype=torch.float32, device="cuda") if lse else None
    ws = kv.alloc_attn_prefill_workspace(d, N)
    ws.fill_(255)
    kv.gdn_attn_prefill(d, layer, i32(cu), q, pool.k, pool.v, i32(pool.table if table is None else table),
                        i32(pool.lens if lens is None else lens), None if pre is None else i32(pre), causal,
                        D ** -0.5 if scale is None else scale, out, ls, ws)
    return out, ls


def check(pool, cu, q, out, lse, causal, pre=None, layer=0, slot0=0, scale=None):
    m = int(cu[-1])
    args = (pool.table, pool.lens, pre, causal, pool.D ** -0.5 if scale is None else scale, slot0)
    k, v = np.nan_to_num(f64(pool.k[layer])), np.nan_to_num(f64(pool.v[layer]))
    ref, ref_lse = O.attention(cu, f64(q)[:m], k, v, *args)
    mag, _ = O.attention(cu, f64(q)[:m], k, np.abs(v), *args)
    got = f64(out)[:m]
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > ROUND[pool.dtype] * (mag + np.abs(ref)) + 2e-4 * mag
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - ref).max())
    assert (out[m:] == 9.0).all()
    if lse is not None:
        empty = np.isinf(ref_lse)
        got = f64(lse)[:m]
        assert np.array_equal(np.isneginf(got), empty)
        assert np.abs(got[~empty] - ref_lse[~empty]).max(initial=0) <= 1e-4
        assert (lse[m:] == 9.0).all()


def run_case(seed, new, lens, Hq, causal=True, prefixes=(), pre=None, layer=0, slot0=0, scale=None, spare_rows=0, wide=False,
             **pool_args):
    """new[b] queries of slots with lens[b] tokens in all."""
    pool = Pool(seed, [5] * slot0 + list(lens) + list(prefixes), **pool_args)
    cu = np.concatenate([[0], np.cumsum(new)])
    N = int(cu[-1]) + spare_rows
    q = pool.gauss((N, Hq, pool.D), 2.0)
    if wide:                                   # queries within a projection's rows
        x = pool.nan((N, (Hq + 3) * pool.D))
        x[:, pool.D:(Hq + 1) * pool.D] = q.flatten(1)
        q = x[:, pool.D:(Hq + 1) * pool.D].unflatten(1, (Hq, pool.D))
    q[int(cu[-1]):] = NAN
    out, lse = attend(pool, cu, q, causal, pre, layer, slot0, scale)
    check(pool, cu, q, out, lse, causal, pre, layer, slot0, scale)
    return pool, cu, q, out, lse


LENS = [1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("G", [1, 4])
def test_prompts_around_the_tiles(D, dtype, G):
    run_case(1, LENS, LENS, 2 * G, D=D, dtype=dtype)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64)])
def test_chunks_behind_cached_tokens(causal, dtype, D):
    """Single tokens, chunks and whole prompts; empty sequences; pages that end inside a tile."""
    run_case(2, [1, 5, 0, 64, 130, 0, 1, 33], [700, 5, 40, 300, 517, 0, 1, 129], 6, causal, D=D, dtype=dtype, spare_rows=3)


@pytest.mark.parametrize("ps", [16, 32, 48, 64, 80, 128, 208, 256, 1024])
@pytest.mark.parametrize("order", ["nhd", "hnd", "mixed"])
def test_page_sizes_and_orders(ps, order):
    run_case(3, [20, 1, 70], [ps + 1, 130, 333], 4, True, prefixes=[ps - 1], pre=[3, -1, 3], ps=ps, order=order, D=128,
             layers=2, layer=1)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (6, 2), (5, 1), (24, 3), (20, 1), (64, 2), (128, 1), (254, 2)])
def test_heads(Hq, Hkv):
    run_case(4, [40, 1, 3], [60, 150, 3], Hq, Hkv=Hkv, D=64)
    run_case(5, [3, 17], [129, 200], Hq, False, Hkv=Hkv, D=64, wide=True)


@pytest.mark.parametrize("plen", [0, 1, 16, 127, 128, 129, 400])
@pytest.mark.parametrize("causal", [False, True])
def test_prefix_lengths(plen, causal):
    run_case(6, [3, 70, 1, 17], [3, 90, 0, 260], 4, causal, prefixes=[plen], pre=[4, 4, 4, 4], D=128, slot0=0)
    run_case(7, [3, 70], [3, 90], 4, causal, prefixes=[plen, 20], pre=[4, 3], D=64, slot0=1, dtype=HF)


def test_rows_without_keys():
    """Slots shorter than their queries: causal rows before the first token are empty, as are all rows over an
    empty slot; behind a prefix they see the prefix."""
    for causal in (True, False):
        run_case(8, [40, 5, 1, 130], [7, 0, 0, 129], 4, causal, D=128)
        run_case(9, [40, 5, 300], [7, 0, 2], 4, causal, prefixes=[33, 0], pre=[3, 4, 3], D=64)


def test_scales():
    for scale in (0.0, -0.2, 1.5):
        run_case(10, [40, 3], [60, 150], 4, scale=scale, D=64)


def test_without_lse_and_without_work():
    pool = Pool(11, [60, 20])
    q = pool.gauss((30, 4, pool.D), 2.0)
    a, _ = attend(pool, [0, 10, 30], q, True)
    b, none = attend(pool, [0, 10, 30], q, True, lse=False)
    assert none is None and torch.equal(a, b)
    out, lse = attend(pool, [0, 0, 0], q, True)
    assert (out == 9.0).all() and (lse == 9.0).all()


@pytest.mark.parametrize("causal", [False, True])
def test_long_axis_split_over_the_card(causal):
    """Few rows over many keys, and one row: pieces are joined, and give the same bits again."""
    for new, lens, Hq in (([1], [30011], 8), ([5, 1], [9000, 30000], 8), ([70], [20000], 2)):
        pool, cu, q, out, lse = run_case(12, new, lens, Hq, causal, ps=64, D=128)
        for _ in range(3):
            again = attend(pool, cu, q, causal)
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_long_prompts():
    """Many row blocks of several heads, whose items end anywhere in a CTA's stretch."""
    for D, Hq, Hkv in ((128, 8, 2), (64, 6, 6)):
        pool = Pool(13, [2500, 37, 1700, 400], D=D, Hkv=Hkv, ps=64)
        cu = np.concatenate([[0], np.cumsum([2500, 37, 900, 399])])
        q = pool.gauss((int(cu[-1]), Hq, D), 2.0)
        out, lse = attend(pool, cu, q, True)
        again = attend(pool, cu, q, True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
        for b in range(4):
            lo, hi, n = int(cu[b]), int(cu[b + 1]), int(pool.lens[b])
            at = torch.from_numpy(pool.table[b, :-(-n // 64)]).cuda()
            k, v = (x[0, at].flatten(0, 1)[:n].double() for x in (pool.k, pool.v))
            mask = torch.ones((hi - lo, n), dtype=torch.bool, device="cuda").tril(n - (hi - lo))
            for h in range(Hq):
                x = (q[lo:hi, h].double() @ k[:, h * Hkv // Hq].T * D ** -0.5).masked_fill(~mask, float("-inf"))
                w, vh = torch.softmax(x, 1), v[:, h * Hkv // Hq]
                ref, mag = w @ vh, w @ vh.abs()
                assert ((out[lo:hi, h].double() - ref).abs() <= ROUND[BF] * (mag + ref.abs()) + 2e-4 * mag).all()
                assert (lse[lo:hi, h].double() - torch.logsumexp(x, 1)).abs().max() <= 1e-4


def test_one_call_or_two():
    """A prompt in two chunks gives what it gives in one, up to the rounding of either."""
    pool = Pool(14, [333], D=64)
    q = pool.gauss((333, 4, 64), 2.0)
    whole, whole_lse = attend(pool, [0, 333], q, True)
    first, lse0 = attend(pool, [0, 200], q[:200].contiguous(), True, lens=[200])
    second, lse1 = attend(pool, [0, 133], q[200:].contiguous(), True)
    assert (torch.cat([lse0, lse1]) - whole_lse).abs().max() <= 2e-4
    check(pool, [0, 333], q, torch.cat([first, second]), None, True)
    check(pool, [0, 333], q, whole, whole_lse, True)


def test_peaked_and_growing_scores():
    """Scores that rise by hundreds along the keys (the running maximum moves in every tile) and fall."""
    for sign in (1.0, -1.0):
        pool = Pool(15, [900, 300], D=128)
        ramp = torch.linspace(0.0, 40.0, 900, device="cuda") * sign
        for s in range(2):
            n = int(pool.lens[s])
            for i in range(n):
                pool.k[0, pool.table[s, i // 16], i % 16, :, 0] = ramp[i].item()
        q = pool.gauss((1200, 4, 128), 1.0)
        q[:, :, 0] = 8.0
        cu = [0, 900, 1200]
        out, lse = attend(pool, cu, q, True, scale=1.0)
        m = f64(q)
        assert np.isfinite(m).all()
        k, v = np.nan_to_num(f64(pool.k[0])), np.nan_to_num(f64(pool.v[0]))
        args = (pool.table, pool.lens, None, True, 1.0)
        ref, ref_lse = O.attention(cu, m, k, v, *args)
        mag, _ = O.attention(cu, m, k, np.abs(v), *args)
        # scores of up to 330: their f32 sums of 128 products are off by 128 * 2^-24 of sum |q k|, at most 6.2e-3
        slack = 128 * 2.0 ** -24 * (8.0 * 40.0 + 128 * 4.0)
        assert (np.abs(f64(out) - ref) <= ROUND[BF] * (mag + np.abs(ref)) + 2 * slack * mag).all()
        assert np.abs(f64(lse) - ref_lse).max() <= slack + 1e-4


def test_what_no_row_sees_may_hold_anything():
    """NaN and infinities behind a slot's tokens (Pool fills them with NaN), in rows behind the last sequence, in
    other slots' pages; and in keys that lie ahead of a row."""
    pool = Pool(16, [70, 33, 200], D=128, ps=32)
    q = pool.gauss((40, 4, 128), 2.0)
    cu = [0, 20, 30, 40]
    want = attend(pool, cu, q, True)
    junk = Pool(16, [70, 33, 200], D=128, ps=32)
    for x in (junk.k, junk.v):
        x[torch.isnan(x)] = float("inf")
    q2 = torch.cat([q, torch.full((5, 4, 128), float("inf"), dtype=BF, device="cuda")])
    got = attend(junk, cu, q2, True)
    assert all(torch.equal(a, b[:40]) for a, b in zip(want, got))
    page, row = pool.table[0, 69 // 32], 69 % 32       # the last token's key: seen by the last row alone
    for bad in (NAN, float("inf"), -float("inf")):
        pool.k[0, page, row] = bad
        got = attend(pool, cu, q, True)
        assert all(torch.equal(a[:19], b[:19]) and torch.equal(a[20:], b[20:]) for a, b in zip(want, got)), bad


@pytest.mark.parametrize("page", [-1, 1 << 27])
def test_a_bad_page_leaves_the_other_sequences_alone(page):
    pool = Pool(17, [40, 300, 17, 130], D=64)
    q = pool.gauss((60, 4, 64), 2.0)
    cu = [0, 20, 30, 40, 60]
    want = attend(pool, cu, q, True)
    table = pool.table.copy()
    table[1, 0] = page
    got = attend(pool, cu, q, True, table=table)
    assert gdn.gdn_device_status(clear=True) == kv.DEVERR_KV_PAGE
    assert all(torch.equal(a[:20], b[:20]) and torch.equal(a[30:], b[30:]) for a, b in zip(want, got))


def test_status():
    pool = Pool(18, [40, 30, 20], D=64)
    q = pool.gauss((30, 4, 64), 2.0)
    cu = [0, 10, 20]
    want = attend(pool, cu, q, True, pre=[2, -1])
    for lens, bit in (([40, -1, 20], kv.DEVERR_KV_LEN), ([40, 1 << 20, 20], kv.DEVERR_KV_LEN)):
        got = attend(pool, cu, q, True, pre=[2, -1], lens=lens)
        assert gdn.gdn_device_status(clear=True) == bit
        assert torch.equal(got[0][:10], want[0][:10]) and (got[0][10:20] == 0).all() and torch.isneginf(got[1][10:20]).all()
    got = attend(pool, cu, q, True, pre=[2, 3])
    assert gdn.gdn_device_status(clear=True) == kv.DEVERR_KV_SLOT and torch.equal(got[0], want[0])
    for bad in ([0, 10, 31], [1, 10, 20], [0, 20, 10], [0, -1, 20], [0, 1 << 30, 20]):
        got = attend(pool, bad, q, True)
        assert gdn.gdn_device_status(clear=True) == gdn.DEVERR_SEQLENS, bad
        assert (got[0] == 9.0).all() and (got[1] == 9.0).all()


@pytest.mark.parametrize("B", [33, 513, 1100])
def test_many_sequences(B):
    """Batches of more sequences than a warp, a step of the plan, and two steps of a search."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 40, B)
    new = np.where(rng.random(B) < 0.3, 0, rng.integers(0, 4, B))
    run_case(19, new, lens, 2, True, prefixes=[30], pre=np.where(rng.random(B) < 0.5, B, -1), Hkv=1, D=64)
    run_case(20, np.minimum(new, 1), lens, 2, False, Hkv=1, D=64)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,dtype,ps", [(64, HF, 16), (64, BF, 48), (128, BF, 64), (128, HF, 80)])
def test_few_rows(G, causal, D, dtype, ps):
    """At most about eight rows a sequence and kv head: single tokens and a few more, beside sequences without any,
    over lengths around the units of keys, behind prefixes and without, with more tokens than keys."""
    lens = [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 129, 0, 2, 517, 40]
    new = [1] * len(lens)
    new[3], new[5], new[12], new[13], new[8] = 0, 2, 1, 2, 0
    if G <= 2:
        new[10] = 3
    pre = [16, -1, 17, 16, -1] * 3 + [18]
    run_case(30 + G, new, lens, 2 * G, causal, prefixes=[33, 0, 300], pre=pre, D=D, dtype=dtype, ps=ps, spare_rows=2)
    run_case(50 + G, [1, 2, 0, 5] if G == 1 else [1, 0, 1, 1], [1, 1, 0, 3], G, causal, Hkv=1, D=D, dtype=dtype, ps=ps)
    pool, cu, q, out, lse = run_case(70 + G, [1, 1], [3000, 7], 3 * G, causal, Hkv=3, D=D, dtype=dtype, ps=ps, order="hnd")
    again = attend(pool, cu, q, causal)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("ps", [16, 64])
def test_few_rows_of_many_sequences(ps):
    """More pieces than workers, and stretches of whole items."""
    rng = np.random.default_rng(ps)
    lens = rng.integers(0, 200, 400)
    run_case(80, np.ones(400, dtype=int), lens, 8, False, Hkv=8, D=64, ps=ps, dtype=HF)
    run_case(81, np.ones(400, dtype=int), lens, 8, True, Hkv=2, D=128, ps=ps, prefixes=[70], pre=[400] * 400)


def test_what_few_rows_do_not_see_may_hold_anything():
    pool = Pool(82, [70, 33, 200], D=128, ps=32)
    q = pool.gauss((4, 4, 128), 2.0)
    cu = [0, 2, 3, 4]
    want = attend(pool, cu, q, True)
    page, row = pool.table[0, 69 // 32], 69 % 32       # the last token's key: seen by the last row alone
    for bad in (NAN, float("inf"), -float("inf")):
        pool.k[0, page, row] = bad
        got = attend(pool, cu, q, True)
        assert all(torch.equal(a[:1], b[:1]) and torch.equal(a[2:], b[2:]) for a, b in zip(want, got)), bad
    table = pool.table.copy()
    table[1, 1] = 1 << 27
    got = attend(pool, cu, q, True, table=table)
    assert gdn.gdn_device_status(clear=True) == kv.DEVERR_KV_PAGE
    assert all(torch.equal(a[:1], b[:1]) and torch.equal(a[3:], b[3:]) for a, b in zip(want, got))


@pytest.mark.parametrize("D,Hq,Hkv,lens,new,plen,causal", [
    (128, 16, 4, [40000], [300], 0, True), (128, 16, 4, [21000, 20500], [290, 512], 0, True),
    (64, 16, 8, [33000], [513], 0, False), (64, 12, 4, [17000, 16801, 17300], [200, 333, 257], 65000, True),
    (128, 6, 2, [70001], [170], 0, True)])
def test_late_chunks(D, Hq, Hkv, lens, new, plen, causal):
    """Few items over many keys, each cut over several CTAs, against float64 row by row."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(D + len(lens))
    ps, G = 64, Hq // Hkv
    slots = lens + ([plen] if plen else [])
    pages = [-(-n // ps) for n in slots]
    ids = torch.randperm(sum(pages), generator=gen, device="cuda").int()
    table = torch.full((len(slots), max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = ids[at:at + n]
        at += n
    k, v = (torch.empty((1, sum(pages), ps, Hkv, D), dtype=BF, device="cuda").normal_(generator=gen) for _ in range(2))
    cu = np.concatenate([[0], np.cumsum(new)])
    q = torch.empty((int(cu[-1]), Hq, D), dtype=BF, device="cuda").normal_(0.0, 2.0, generator=gen)
    d = kv.make_kv_dims(len(lens), 1, Hq, Hkv, D, ps, sum(pages), max(pages), len(slots))
    ws = kv.alloc_attn_prefill_workspace(d, q.shape[0])
    pre = i32([len(lens)] * len(lens)) if plen else None
    runs = []
    for fill in (255, 0):
        ws.fill_(fill)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
        kv.gdn_attn_prefill(d, 0, i32(cu), q, k, v, table, i32(slots), pre, causal, D ** -0.5, out, lse, ws)
        runs.append((out, lse))
    assert gdn.gdn_device_status(clear=True) == 0
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    for b, n in enumerate(lens):
        order = ([len(lens)] if plen else []) + [b]
        kb, vb = (torch.cat([x[0, table[s, :pages[s]].long()].flatten(0, 1)[:slots[s]] for s in order]).double() for x in (k, v))
        lo, hi = int(cu[b]), int(cu[b + 1])
        mask = torch.ones((hi - lo, kb.shape[0]), dtype=torch.bool, device="cuda")
        if causal:
            mask = mask.tril(kb.shape[0] - (hi - lo))
        for h in range(Hq):
            x = (q[lo:hi, h].double() @ kb[:, h // G].T * D ** -0.5).masked_fill(~mask, float("-inf"))
            w = torch.softmax(x, 1)
            ref, mag = w @ vb[:, h // G], w @ vb[:, h // G].abs()
            assert ((out[lo:hi, h].double() - ref).abs() <= ROUND[BF] * (mag + ref.abs()) + 2e-4 * mag).all(), (b, h)
            assert (lse[lo:hi, h].double() - torch.logsumexp(x, 1)).abs().max() <= 1e-4


@pytest.mark.parametrize("new,lens,G", [([5], [2], 1), ([200], [60], 4), ([300, 2], [290, 1], 2), ([3, 4], [1, 300], 2), ([200], [199], 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_without_keys_do_not_meet_values_of_others(D, new, lens, G):
    """Rows before the slot's first token get 0 and -inf, also where the value of a token that others see is not finite."""
    pool = Pool(83, lens, D=D, ps=32, Hkv=1)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = pool.gauss((int(cu[-1]), G, D), 2.0)
    for bad in (NAN, float("inf")):
        for s, n in enumerate(lens):
            pool.v[0, pool.table[s, (n - 1) // 32], (n - 1) % 32] = bad
        out, lse = attend(pool, cu, q, True)
        for s, n in enumerate(lens):
            none = slice(int(cu[s]), int(cu[s]) + max(0, new[s] - n))
            assert (out[none] == 0).all() and torch.isneginf(lse[none]).all()
            own = int(cu[s + 1]) - 1
            assert not torch.isfinite(out[own]).any() and torch.isfinite(lse[own]).all()


@pytest.mark.parametrize("length", [40, 128, 129, 161, 300, 1000, 2049, 20000, 60001])
@pytest.mark.parametrize("D,Hq,Hkv,B", [(128, 8, 1, 1), (64, 3, 3, 1), (128, 32, 8, 1), (64, 32, 4, 2), (128, 18, 9, 1), (64, 16, 16, 2)])
def test_a_token_in_many_pieces(D, Hq, Hkv, B, length):
    """Single tokens, whose keys are dealt to so many warps that a few or all of the join's CTAs share their pieces."""
    lens = [length, 77][:B]
    pool, cu, q, out, lse = run_case(84, [1] * B, lens, Hq, D=D, Hkv=Hkv, ps=64)
    again, lse2 = attend(pool, cu, q, True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
