"""Reserve, append and attention one after the other where reserve has no room for a sequence: the tokens that are
cached stay as they are, in that sequence and in those that share its pages, and the other sequences' results are
theirs alone.

Heads are neither normed nor rotated here, so what append writes is its input bit for bit and the whole pool has
one right answer.  Attention's tolerances are those of test_gpu_kv_prefill.py."""
import numpy as np
import pytest
import torch

from kv_util import ROUND, f64, i32
from oracle import prompt_oracle as O
from speculative_decode_verify_gdn_gb300 import gdn, kv
from speculative_decode_verify_gdn_gb300.build import build_library
from speculative_decode_verify_gdn_gb300.kv_runtime import PagedCache

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
LEN, PAGE, FULL, SHARED = kv.DEVERR_KV_LEN, kv.DEVERR_KV_PAGE, kv.DEVERR_KV_FULL, kv.DEVERR_KV_SHARED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    build_library()
    kv.load_library()
    gdn.gdn_device_status(clear=True)
    yield
    assert gdn.gdn_device_status(clear=True) == 0


B, PS, LAYERS, HKV = 5, 16, 2, 2


class Run:
    """Sequences 0 and 1 share two whole pages, 4 has a prefix; `free` pages are left."""

    def __init__(self, dtype, D, G, free):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(5)
        self.dtype, self.D, self.Hq = dtype, D, G * HKV
        self.cache = c = PagedCache.create(B, 1, self.Hq, HKV, D, PS, n_pages=7 + free, max_pages=4, n_prefixes=1, n_layers=LAYERS,
                                           dtype=dtype)
        c.k.fill_(float("nan")), c.v.fill_(float("nan"))
        self.plain = kv.make_rope(D)
        self.fill([32, 0, 7, 20, 3, 11])
        c.fork(i32([0, 0, 2, 3, 4, 5]))
        c.prefix_of[4] = 5
        assert gdn.gdn_device_status(clear=True) == 0
        assert int((c.ref == 0).sum()) == free and c.table[0, :2].tolist() == c.table[1, :2].tolist()

    def rows(self, *shape):
        return torch.empty(shape, dtype=self.dtype, device="cuda").normal_(generator=self.gen)

    def fill(self, lens):
        for slot, n in enumerate(lens):
            if n:
                self.cache.append(slot, self.rows(LAYERS, n, HKV, self.D), self.rows(LAYERS, n, HKV, self.D))

    def buffers(self, n):
        q, k, v = (self.rows(LAYERS, n, h, self.D) for h in (self.Hq, HKV, HKV))
        q_out, out = (torch.full_like(q, 5.0) for _ in range(2))
        return q, k, v, q_out, out, torch.full((LAYERS, n, self.Hq), 5.0, device="cuda")

    def step(self, new, cu, bufs):
        q, k, v, q_out, out, lse = bufs
        self.cache.reserve(new)
        for i in range(LAYERS):
            self.cache.append_layer(i, self.plain, cu, q[i], k[i], v[i], q_out[i])
            self.cache.attend_prefill(i, cu, q_out[i], out[i], lse[i])


def bits(t):
    return t.view(torch.int16).clone()


def check(run, asked, cu, before, lens, bufs, refused):
    """After a step that had no room for the sequences in `refused`."""
    c, (q, k, v, q_out, out, lse) = run.cache, bufs
    after = lens.copy()
    for b in range(B):
        if b not in refused:
            after[b] += asked[b]
    assert c.seq_len.tolist() == after.tolist()
    assert c.refused.tolist()[:B] == [int(lens[b]) if b in refused else -1 for b in range(B)]
    # the pool: what it held, and the tokens of those that got their room
    table = c.table.cpu().numpy()
    for was, now, new in zip(before, (c.k, c.v), (k, v)):
        want = was.clone()
        for b in range(B):
            for j in range(0 if b in refused else asked[b]):
                at = int(lens[b]) + j
                want[:, table[b, at // PS], at % PS] = bits(new[:, int(cu[b]) + j])
        assert torch.equal(bits(now), want)
    pre = [-1, -1, -1, -1, 5]
    for i in range(LAYERS):
        kc, vc = np.nan_to_num(f64(c.k[i])), np.nan_to_num(f64(c.v[i]))
        ref, ref_lse = O.attention(cu, f64(q[i]), kc, vc, table, after, pre, True, run.D ** -0.5)
        mag, _ = O.attention(cu, f64(q[i]), kc, np.abs(vc), table, after, pre, True, run.D ** -0.5)
        for b in range(B):
            at = slice(int(cu[b]), int(cu[b + 1]))
            if b in refused:
                assert (q_out[i, at] == 5.0).all() and (out[i, at] == 0.0).all() and torch.isneginf(lse[i, at]).all()
                continue
            assert torch.equal(q_out[i, at], q[i, at])
            assert (np.abs(f64(out[i])[at] - ref[at]) <= ROUND[run.dtype] * (mag[at] + np.abs(ref[at])) + 2e-4 * mag[at]).all()
            assert (np.abs(f64(lse[i])[at] - ref_lse[at]) <= 1e-4).all()


CASES = {                       # free pages, tokens asked for, heads to a kv head, who is refused, status
    "full": (1, [17, 0, 5, 3, 1], 4, [0], FULL),
    "full, sequences behind it too": (1, [17, 4, 5, 13, 14], 4, [0, 1, 3, 4], FULL),
    "full, few rows": (0, [1, 0, 1, 1, 1], 2, [0], FULL),
    "columns": (9, [33, 0, 5, 3, 13], 4, [0], FULL),
    "out of range": (9, [-1, 0, 5, 3, 1], 4, [0], LEN),
    "a last page that is shared": (9, [20, 2, 5, 3, 1], 4, [2], SHARED),
}


@pytest.mark.parametrize("dtype,D", [(BF, 128), (HF, 64)])
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_cached_tokens_stay(name, captured, dtype, D):
    free, asked, G, refused, status = CASES[name]
    run = Run(dtype, D, G, free)
    c = run.cache
    if status == SHARED:
        c.ref[int(c.table[2, 0])] += 1
    rows = [max(n, 3 if n < 0 else 0) for n in asked]        # (a call out of range brings three rows all the same)
    cu = np.concatenate([[0], np.cumsum(rows)])
    new, bounds = i32([0] * B), i32([0] * (B + 1))
    bufs = run.buffers(int(cu[-1]))
    run.step(new, bounds, bufs)                              # nothing asked for, nothing done
    assert gdn.gdn_device_status(clear=True) == 0 and (bufs[4] == 5.0).all()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run.step(new, bounds, bufs)
    new.copy_(i32(asked)), bounds.copy_(i32(cu))
    before, lens = (bits(c.k), bits(c.v)), c.seq_len.cpu().numpy().astype(np.int64)
    torch.cuda.synchronize()
    graph.replay() if captured else run.step(new, bounds, bufs)
    assert gdn.gdn_device_status(clear=True) == status | LEN
    check(run, rows, cu, before, lens, bufs, refused)


def test_asked_again():
    """A sequence that there was no room for gets its tokens once pages are free; one that went on by verify rounds
    instead is attended again."""
    run = Run(BF, 64, 2, 0)
    c = run.cache
    asked = [5, 0, 1, 0, 0]
    cu = np.concatenate([[0], np.cumsum(asked)])
    bufs = run.buffers(6)
    before, lens = (bits(c.k), bits(c.v)), c.seq_len.cpu().numpy().astype(np.int64)
    run.step(i32(asked), i32(cu), bufs)
    assert gdn.gdn_device_status(clear=True) == FULL | LEN
    check(run, asked, cu, before, lens, bufs, [0])
    c.fork(i32([0, 1, 2, -1, 4, 5]))                         # sequence 3's two pages are free
    asked = [5, 0, 0, 1, 0]
    cu = np.concatenate([[0], np.cumsum(asked)])
    bufs = run.buffers(6)
    before, lens = (bits(c.k), bits(c.v)), c.seq_len.cpu().numpy().astype(np.int64)
    run.step(i32(asked), i32(cu), bufs)
    assert gdn.gdn_device_status(clear=True) == 0
    check(run, asked, cu, before, lens, bufs, [])
    run.cache.reserve(i32([0, 1000, 0, 0, 0]))
    assert gdn.gdn_device_status(clear=True) == FULL and c.refused.tolist()[1] == 32
    c.fork(i32([0, 1, 2, -1, 4, 5]))                         # sequence 3's page again
    c.reserve(i32([0, 1000, 0, 0, 0]))
    one = run.rows(LAYERS, B, 1, HKV, run.D)
    c.commit(i32([0, 1, 0, 0, 0]), one, one)
    q = run.rows(2, run.Hq, run.D)
    out, lse = torch.empty_like(q), torch.empty((2, run.Hq), device="cuda")
    c.attend_prefill(0, i32([0, 0, 2, 2, 2, 2]), q, out, lse)
    assert gdn.gdn_device_status(clear=True) == FULL         # (the second refusal alone)
    assert torch.isfinite(lse).all() and (out != 0).any()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_seq,n_pages", [(3, 4), (700, 900), (700, 20000)])
def test_what_reserve_notes(n_seq, n_pages, in_place):
    """Entries of the call's own slots, with and without room for all of them in one step of the plan."""
    rng = np.random.default_rng(n_seq + n_pages)
    slot0, slots, max_pages = 2, n_seq + 5, 6
    lens = rng.integers(0, 3 * PS, slots)
    table, cnt = np.full((slots, max_pages), -1), np.zeros(n_pages, dtype=np.int64)
    ids = iter(rng.permutation(n_pages))
    for s in range(slots):
        for c in range(-(-int(lens[s]) // PS)):
            page = next(ids, None)
            if page is None:
                lens[s] = c * PS
                break
            table[s, c], cnt[page] = page, 1
    asked = rng.integers(-1, 60, n_seq)
    asked[rng.random(n_seq) < 0.3] = 0
    t, n, r = O.reserve(asked, table, lens, cnt, PS, slot0)
    d = kv.make_kv_dims(n_seq, 1, 2, 2, 64, PS, n_pages, max_pages, slots, slot0)
    args = [i32(x) for x in (table, lens, cnt)]
    outs = args if in_place else [torch.full_like(x, 9) for x in args]
    refused = torch.full((slots,), 9, dtype=torch.int32, device="cuda")
    kv.gdn_kv_reserve(d, i32(asked), args[0], outs[0], args[1], (outs[1], refused), args[2], outs[2], kv.alloc_kv_workspace(d))
    gdn.gdn_device_status(clear=True)
    assert all(np.array_equal(x.cpu().numpy(), want) for x, want in zip(outs, (t, n, r)))
    want = np.full(slots, 9)
    mine = slice(slot0, slot0 + n_seq)
    want[mine] = np.where((asked != 0) & (n[mine] == lens[mine]), lens[mine], -1)
    assert np.array_equal(refused.cpu().numpy(), want)
