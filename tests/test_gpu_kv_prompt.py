"""Prompts and verify rounds of a small stack of attention layers through PagedCache, as a model runs them: reserve, then
layer by layer append and prefill attention; windows normed and rotated, attended, committed - against float64
attention over each sequence's whole history, computed from the projections alone.

Tolerances.  Rotated queries and keys are rounded once (u of the type, relative), which moves a score of queries and
keys by at most 2 u sum |q_i k_i| scale; with heads normed to length sqrt(D) that sum is at most D by Cauchy-Schwarz times
the weights' 1.6^2, so a score moves by up to 2 u 1.6^2 sqrt(D) =: s and a weight by the factor e^(2 s) at most.  On top
of that come the attention's own u (A + |ref|) + 2e-4 A (test_gpu_kv_attn.py), A = sum w |v|."""
import math

import numpy as np
import pytest
import torch

from kv_util import ROUND, i32
from speculative_decode_verify_gdn_gb300 import gdn, kv, rope
from speculative_decode_verify_gdn_gb300.build import build_library
from speculative_decode_verify_gdn_gb300.kv_runtime import PagedCache

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


class Layer:
    def __init__(self, gen, Hq, Hkv, D, dtype, rot, inter):
        def weight():
            return torch.empty(D, device="cuda").uniform_(-0.6, 0.6, generator=gen)
        self.Hq, self.Hkv, self.D, self.dtype, self.gen = Hq, Hkv, D, dtype, gen
        self.radians = rope.frequencies(rot, scaling="ramp", factor=4.0, trained=512)
        self.w, self.inter = (weight(), weight()), inter
        self.rope = kv.make_rope(D, self.radians, inter, q_weight=self.w[0], k_weight=self.w[1], weight_offset=1.0)

    def project(self, n):
        """Rows of a projection, and its parts q, k, v [n, heads, D]."""
        x = torch.empty((n, (self.Hq + 2 * self.Hkv) * self.D), dtype=self.dtype, device="cuda").normal_(generator=self.gen)
        q, k, v = x.split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], 1)
        return q.view(n, self.Hq, self.D), k.view(n, self.Hkv, self.D), v.view(n, self.Hkv, self.D)

    def turned(self, x, which, positions):
        """x [n, H, D] in float64, normed and rotated."""
        x = x.double()
        x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * (1.0 + self.w[which].double())
        half = self.radians.numel()
        z = x[..., :2 * half].unflatten(-1, (half, 2) if self.inter else (2, half))
        a, b = (z[..., 0], z[..., 1]) if self.inter else (z[..., 0, :], z[..., 1, :])
        phi = (positions.double()[:, None] * self.radians.cuda())[:, None]
        y = torch.stack([a * phi.cos() - b * phi.sin(), b * phi.cos() + a * phi.sin()], -1 if self.inter else -2).flatten(-2)
        return torch.cat([y, x[..., 2 * half:]], -1)


class History:
    """What a sequence's tokens were, for the reference: keys (rotated) and values of one layer in float64."""

    def __init__(self, k=None, v=None):
        self.k, self.v = k, v

    def add(self, k, v):
        return History(k if self.k is None else torch.cat([self.k, k]), v if self.v is None else torch.cat([self.v, v]))


def expect(layer, q, h, seen):
    """out and A of queries [n, Hq, D] (rotated, float64) over a history, row i seeing seen[i] (a bool mask [n, keys])."""
    G = layer.Hq // layer.Hkv
    x = torch.einsum("nhd,khd->hnk", q, h.k.repeat_interleave(G, 1)) * layer.D ** -0.5
    w = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
    v = h.v.repeat_interleave(G, 1)
    return torch.einsum("hnk,khd->nhd", w, v), torch.einsum("hnk,khd->nhd", w, v.abs())


def close(layer, got, ref, mag):
    u = ROUND[layer.dtype]
    s = 2 * u * 1.6 ** 2 * math.sqrt(layer.D)
    assert ((got.double() - ref).abs() <= u * (mag + ref.abs()) + (2e-4 + math.expm1(2 * s)) * mag).all(), \
        ((got.double() - ref).abs() / mag).max()


def causal(n, keys):
    return torch.ones((n, keys), dtype=torch.bool, device="cuda").tril(keys - n)


@pytest.mark.parametrize("dtype,D,inter", [(BF, 128, False), (HF, 64, True)])
def test_prompts_and_rounds(dtype, D, inter):
    B, K, Hq, Hkv, ps, layers = 3, 5, 6, 2, 16, 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rng = np.random.default_rng(1)
    L = [Layer(gen, Hq, Hkv, D, dtype, D // 2, inter) for _ in range(layers)]
    cache = PagedCache.create(B, K, Hq, Hkv, D, ps, n_pages=200, max_pages=40, n_prefixes=1, n_layers=layers, dtype=dtype)
    prefix = [History() for _ in L]
    own = [[History() for _ in range(B)] for _ in L]

    def feed(new, slot0, base):
        """A chunk of new[i] tokens of each sequence from slot0 on, whose tokens begin at position base."""
        cu = np.concatenate([[0], np.cumsum(new)])
        start = cache.seq_len[slot0:slot0 + len(new)].tolist()
        cache.reserve(i32(new), slot0)
        for i, layer in enumerate(L):
            q, k, v = layer.project(int(cu[-1]) + 4)             # (four rows of padding)
            q_out = torch.empty((q.shape[0], Hq, D), dtype=dtype, device="cuda")
            out, lse = torch.full_like(q_out, 7.0), torch.empty((q.shape[0], Hq), device="cuda")
            cache.append_layer(i, layer.rope, i32(cu), q, k, v, q_out, slot0)
            cache.attend_prefill(i, i32(cu), q_out, out, lse, slot0)
            assert (out[int(cu[-1]):] == 7.0).all()
            for b, n in enumerate(new):
                at = slice(int(cu[b]), int(cu[b + 1]))
                pos = base + start[b] + torch.arange(n, device="cuda")
                mine = prefix[i] if slot0 == B else own[i][slot0 + b]
                mine = mine.add(layer.turned(k[at], 1, pos), v[at].double())
                if slot0 == B:
                    prefix[i], seen = mine, mine
                else:
                    own[i][slot0 + b], seen = mine, prefix[i].add(mine.k, mine.v)
                if n:
                    close(layer, out[at], *expect(layer, layer.turned(q[at], 0, pos), seen, causal(n, seen.k.shape[0])))

    feed([77], B, 0)                                             # the shared prompt, in two chunks
    feed([60], B, 0)
    cache.prefix_of.fill_(B)
    feed([33, 1, 150], 0, 137)                                   # prompts, then chunks of some of them, then one alone
    feed([20, 0, 1], 0, 137)
    feed([17], 1, 137)
    for r in range(3):                                           # verify rounds of trees
        parent = np.stack([[t - 1 if t < 3 else 1 for t in range(K)]] * B) if r else None
        accept = rng.integers(1, K + 1, B)
        k_win, v_win = (torch.empty((layers, B, K, Hkv, D), dtype=dtype, device="cuda") for _ in range(2))
        lens = cache.seq_len.tolist()
        depth = np.array([[0, 1, 2, 2, 2]] * B) if r else np.array([list(range(K))] * B)
        paths = [[[t for t in range(K) if t == n or (t < n and (parent is None or (t < 2 and (n != 1 or t == 0))))] for n in range(K)]] * B
        for i, layer in enumerate(L):
            q, k, v = (x.unflatten(0, (B, K)) for x in layer.project(B * K))
            q_out = torch.empty((B, K, Hq, D), dtype=dtype, device="cuda")
            out = torch.empty_like(q_out)
            par = None if parent is None else i32(parent)
            cache.rope(layer.rope, q, k, v, q_out, k_win[i], v_win[i], parent=par)
            cache.attend(i, q_out, k_win[i], v_win[i], out, parent=par)
            for b in range(B):
                pos = torch.from_numpy(137 + lens[b] + depth[b]).cuda()
                kt, vt = layer.turned(k[b], 1, pos), v[b].double()
                seen = prefix[i].add(own[i][b].k, own[i][b].v).add(kt, vt)
                mask = torch.ones((K, seen.k.shape[0]), dtype=torch.bool, device="cuda")
                mask[:, -K:] = False
                for n in range(K):
                    mask[n, [seen.k.shape[0] - K + t for t in paths[b][n]]] = True
                close(layer, out[b], *expect(layer, layer.turned(q[b], 0, pos), seen, mask))
                kept = paths[b][accept[b] - 1]
                own[i][b] = own[i][b].add(kt[kept], vt[kept])
        cache.commit(i32(accept), k_win, v_win, parent=None if parent is None else i32(parent))
    feed([3, 40, 0], 0, 137)                                     # another chunk behind the drafted tokens
    feed([1, 1, 1], 0, 137)                                      # plain decode
    held = torch.bincount(cache.table[cache.table >= 0].long(), minlength=200)
    assert torch.equal(held, cache.ref.long())


def test_cross_attention_beside_the_sequences():
    """Encoder states of several lengths in the slots; queries of one token and of many, in place of a prompt's."""
    B, Hq, Hkv, D = 4, 4, 4, 64
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    layer = Layer(gen, Hq, Hkv, D, BF, 0, False)                 # no rotation, norms alone
    cache = PagedCache.create(B, 1, Hq, Hkv, D, 48, n_pages=60, max_pages=12)
    lens = [300, 0, 47, 500]
    cu = np.concatenate([[0], np.cumsum(lens)])
    cache.reserve(i32(lens))
    _, k, v = layer.project(int(cu[-1]))
    cache.append_layer(0, layer.rope, i32(cu), None, k, v, None)
    for new in ([1, 1, 1, 1], [200, 7, 0, 64]):
        cq = np.concatenate([[0], np.cumsum(new)])
        q, _, _ = layer.project(int(cq[-1]))
        q_out, out = torch.empty_like(q), torch.empty(q.shape, dtype=BF, device="cuda")
        q_out = torch.empty(q.shape, dtype=BF, device="cuda")
        d = kv.make_kv_dims(q.shape[0], 1, Hq, Hkv, D, 48, 1, 1)
        kv.gdn_attn_rope(d, layer.rope, q[:, None], None, None, None, None, None, None, i32(np.zeros((q.shape[0], 1))), q_out[:, None],
                         None, None)
        cache.attend_prefill(0, i32(cq), q_out, out, causal=False)
        zero = torch.zeros(1, device="cuda")
        for b in range(B):
            at, keys = slice(int(cq[b]), int(cq[b + 1])), slice(int(cu[b]), int(cu[b + 1]))
            if lens[b] == 0:
                assert (out[at] == 0).all()
                continue
            h = History(layer.turned(k[keys], 1, zero.expand(lens[b])), v[keys].double())
            mask = torch.ones((new[b], lens[b]), dtype=torch.bool, device="cuda")
            close(layer, out[at], *expect(layer, layer.turned(q[at], 0, zero.expand(new[b])), h, mask))


def _one_step(cache, layer, cu, new, bufs, stream=None):
    q, k, v, q_out, out, lse = bufs
    cache.reserve(new, stream=stream)
    cache.append_layer(0, layer.rope, cu, q, k, v, q_out, stream=stream)
    cache.attend_prefill(0, cu, q_out, out, lse, stream=stream)


@pytest.mark.parametrize("n", [4, 200])
def test_a_captured_step_serves_other_lengths(n):
    """Reserve, append and attention captured once and replayed with other bounds, in a padded batch of rows; an eager
    run of the same steps gives the same bits.  (4 rows: the kernel for few rows; 200: the tiles.)"""
    B, Hq, Hkv, D = 4, 8, 2, 128
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    layer = Layer(gen, Hq, Hkv, D, BF, 128, False)
    rng = np.random.default_rng(3)
    sides = []
    for _ in range(2):
        c = PagedCache.create(B, 1, Hq, Hkv, D, 16, n_pages=300, max_pages=60)
        c.k.zero_(), c.v.zero_()
        sides.append(c)
    q, k, v = layer.project(n)
    out = [(torch.zeros((n, Hq, D), dtype=BF, device="cuda"), torch.zeros((n, Hq, D), dtype=BF, device="cuda"),
            torch.zeros((n, Hq), device="cuda")) for _ in sides]
    cu, new = i32([0] * (B + 1)), i32([0] * B)
    _one_step(sides[0], layer, cu, new, (q, k, v, *out[0]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _one_step(sides[0], layer, cu, new, (q, k, v, *out[0]))
    for _ in range(5):
        lens = rng.multinomial(rng.integers(0, n + 1), [1 / B] * B)
        q.normal_(generator=gen), k.normal_(generator=gen), v.normal_(generator=gen)
        new.copy_(i32(lens)), cu.copy_(i32(np.concatenate([[0], np.cumsum(lens)])))
        for o in out:
            for x in o:
                x.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        _one_step(sides[1], layer, cu.clone(), new.clone(), (q, k, v, *out[1]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*out))
        assert torch.equal(sides[0].k, sides[1].k) and torch.equal(sides[0].table, sides[1].table)
        assert (out[0][1][int(cu[-1]):] == 5.0).all()


def test_steps_on_streams_of_their_own():
    """Two caches' steps side by side on two streams give what they give one after the other."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    layer = Layer(gen, 8, 2, 64, BF, 64, False)
    lens = [[300, 1, 40, 129], [5, 200, 0, 77]]
    bufs, want = [], []
    for which in lens:
        n = sum(which)
        q, k, v = layer.project(n)
        bufs.append((q, k, v, i32(np.concatenate([[0], np.cumsum(which)])), i32(which)))
    for streams in (None, [torch.cuda.Stream() for _ in lens]):
        caches = [PagedCache.create(4, 1, 8, 2, 64, 16, n_pages=200, max_pages=60) for _ in lens]
        outs = []
        for c in caches:
            c.k.zero_(), c.v.zero_()
        torch.cuda.synchronize()
        for rep in range(3):
            for i, (c, b) in enumerate(zip(caches, bufs)):
                s = None if streams is None else streams[i]
                n = b[0].shape[0]
                with torch.cuda.stream(s):
                    o = tuple(torch.empty(sh, dtype=dt, device="cuda") for sh, dt in
                              (((n, 8, 64), BF), ((n, 8, 64), BF), ((n, 8), torch.float32)))
                _one_step(c, layer, b[3], b[4], (*b[:3], *o), stream=s)
                outs.append(o)
        torch.cuda.synchronize()
        got = [x for o in outs for x in o] + [x for c in caches for x in (c.k, c.v, c.table, c.seq_len, c.ref)]
        if not want:
            want = got
    assert len(want) == len(got) and all(torch.equal(a, b) for a, b in zip(want, got))


def test_no_step_allocates():
    """The calls that a captured step is made of take no memory."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    layer = Layer(gen, 8, 2, 64, BF, 64, False)
    cache = PagedCache.create(2, 1, 8, 2, 64, 16, n_pages=100, max_pages=20)
    q, k, v = layer.project(50)
    o = (torch.empty((50, 8, 64), dtype=BF, device="cuda"), torch.empty((50, 8, 64), dtype=BF, device="cuda"), torch.empty((50, 8), device="cuda"))
    cu, new = i32([0, 30, 50]), i32([30, 20])
    _one_step(cache, layer, cu, new, (q, k, v, *o))
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    _one_step(cache, layer, cu, new, (q, k, v, *o))
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
