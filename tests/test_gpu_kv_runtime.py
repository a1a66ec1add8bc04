"""PagedCache on streams of its own and with several prefixes.  Tolerances are those of
test_gpu_kv_attn.py."""
import numpy as np
import pytest
import torch

from kv_util import ROUND, f64
from oracle import kv_oracle as O
from speculative_decode_verify_gdn_gb300 import gdn, kv
from speculative_decode_verify_gdn_gb300.build import build_library
from speculative_decode_verify_gdn_gb300.kv_runtime import PagedCache

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    build_library()
    kv.load_library()
    gdn.gdn_device_status(clear=True)
    yield
    assert gdn.gdn_device_status(clear=True) == 0


def gauss(*shape):
    return torch.empty(shape, dtype=BF, device="cuda").normal_()


def test_append_on_a_side_stream_beside_a_busy_one():
    """Prompts appended on a stream of their own, while the current one is busy and allocates and
    fills blocks of the sizes that append uses."""
    B, Hkv, D, ps, L = 8, 2, 64, 16, 2
    cache = PagedCache.create(B, 4, 4, Hkv, D, ps, n_pages=400, max_pages=30, n_layers=L)
    prompts = [[gauss(L, n, Hkv, D) for _ in range(2)] for n in (1, 300, 47, 16, 129, 15, 222, 64)]
    busy = gauss(4096, 4096)
    ws = cache.pool_workspace.numel()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for slot, (k, v) in enumerate(prompts):
        busy = (busy @ busy).clamp(-1, 1)
        cache.append(slot, k, v, stream=side)
        junk = [torch.full((1,), -9, dtype=torch.int32, device="cuda"),
                torch.full((ws,), 255, dtype=torch.uint8, device="cuda")]
        del junk
    torch.cuda.synchronize()
    assert gdn.gdn_device_status(clear=True) == 0
    assert cache.seq_len.tolist() == [k.shape[1] for k, _ in prompts]
    for slot, (k, v) in enumerate(prompts):
        n = k.shape[1]
        at = cache.table[slot, :-(-n // ps)].long()
        for x, want in ((cache.k, k), (cache.v, v)):
            assert torch.equal(x[:, at].flatten(1, 2)[:, :n], want)
    held = torch.bincount(cache.table[cache.table >= 0].long(), minlength=400)
    assert torch.equal(held, cache.ref.long()) and int(held.max()) == 1


def test_attention_in_two_streams_at_once():
    """Two caches' calls in flight side by side give what they give one after the other."""
    caches, args = [], []
    for i, (B, n) in enumerate(((4, 3000), (40, 100))):
        c = PagedCache.create(B, 4, 8, 2, 128, 64, n_pages=B * (n // 64 + 2), max_pages=n // 64 + 2)
        for slot in range(B):
            c.append(slot, gauss(1, n - 7 * slot % n, 2, 128), gauss(1, n - 7 * slot % n, 2, 128))
        caches.append(c)
        args.append((gauss(B, 4, 8, 128), gauss(B, 4, 2, 128), gauss(B, 4, 2, 128)))
    want = [torch.empty_like(a[0]) for a in args]
    for c, a, o in zip(caches, args, want):
        c.attend(0, *a, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    got = [[torch.empty_like(a[0]) for _ in range(20)] for a in args]
    torch.cuda.synchronize()
    for i in range(20):
        for c, a, o, s in zip(caches, args, got, streams):
            c.attend(0, *a, o[i], stream=s)
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


@pytest.mark.parametrize("side", [False, True])
def test_fork_across_prefixes(side):
    """Sequences of two prefixes, and one without, forked into each other's slots attend to what the
    sequences they go on from attended to."""
    B, K, Hq, Hkv, D, ps = 6, 3, 4, 2, 64, 16
    cache = PagedCache.create(B, K, Hq, Hkv, D, ps, n_pages=200, max_pages=12, n_prefixes=2)
    lens = [5, 40, 33, 0, 64, 17, 90, 130]
    for slot, n in enumerate(lens):
        if n:
            cache.append(slot, gauss(1, n, Hkv, D), gauss(1, n, Hkv, D))
    cache.prefix_of.copy_(torch.tensor([6, 7, -1, 6, 7, 6], dtype=torch.int32))
    one = [gauss(1, K, h, D) for h in (Hq, Hkv, Hkv)]
    q, kw, vw = (x.expand(B, K, -1, -1).contiguous() for x in one)   # every sequence drafts the same window
    before, after = torch.empty_like(q), torch.empty_like(q)
    cache.attend(0, q, kw, vw, before)
    src = [1, 2, 0, 4, 3, 3]
    s = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    cache.fork(torch.tensor(src + [6, 7], dtype=torch.int32, device="cuda"), stream=s)
    cache.attend(0, q, kw, vw, after, stream=s)
    torch.cuda.synchronize()
    assert cache.prefix_of.tolist() == [7, -1, 6, 7, 6, 6]
    table, n = cache.table.cpu().numpy(), cache.seq_len.cpu().numpy()
    args = (f64(kw), np.abs(f64(vw)), np.nan_to_num(f64(cache.k[0])), np.abs(np.nan_to_num(f64(cache.v[0]))), table, n,
            cache.prefix_of.tolist(), None, None, D ** -0.5)
    mag, _ = O.attention(f64(q), *args)
    want, got = f64(before)[src], f64(after)
    # two roundings of the probabilities and of the output, from different tiles
    assert (np.abs(got - want) <= 2 * (ROUND[BF] * (mag + np.abs(want)) + 2e-4 * mag)).all()
    ref, _ = O.attention(f64(q), f64(kw), f64(vw), np.nan_to_num(f64(cache.k[0])), np.nan_to_num(f64(cache.v[0])), *args[4:])
    assert (np.abs(got - ref) <= ROUND[BF] * (mag + np.abs(ref)) + 2e-4 * mag).all()
