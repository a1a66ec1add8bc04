"""Norms and rotation of calls around the sizes at which a CTA takes more tokens: the bits are those of calls on a part of
the tokens each, and do not depend on what else is in the call."""
import numpy as np
import pytest
import torch

from kv_util import i32
from speculative_decode_verify_gdn_gb300 import gdn, kv, rope
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


def turning(D):
    return kv.make_rope(D, rope.frequencies(D), q_weight=torch.rand(D), k_weight=torch.rand(D))


def rows(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_()


@pytest.mark.parametrize("D,dtype,Hq,Hkv", [(128, BF, 6, 2), (64, HF, 5, 1)])
@pytest.mark.parametrize("B,K", [(1064, 1), (1065, 1), (152, 7), (153, 7), (67, 16), (133, 16), (199, 16), (200, 16), (638, 5), (639, 5)])
def test_windows(D, dtype, Hq, Hkv, B, K):
    r, rng = turning(D), np.random.default_rng(B)
    q, k, v = rows(dtype, B, K, Hq, D), rows(dtype, B, K, Hkv, D), rows(dtype, B, K, Hkv, D)
    lens, win = rng.integers(0, 500, B), rng.integers(0, K + 1, B)
    parent = np.minimum(np.arange(K)[None, :] - 1, rng.integers(-1, K, (B, K)))

    def call(at):
        n = at.stop - at.start
        d = kv.make_kv_dims(n, K, Hq, Hkv, D, 16, 4, 40, dtype=dtype)
        outs = [torch.full_like(x[at].contiguous(), 7.0) for x in (q, k, v)]
        kv.gdn_attn_rope(d, r, q[at], k[at], v[at], i32(lens[at]), None, i32(win[at]), i32(parent[at]), None, *outs)
        return outs

    parts = [call(slice(b, min(B, b + 64 // K + 1))) for b in range(0, B, 64 // K + 1)]
    assert all(torch.equal(a, torch.cat(p)) for a, p in zip(call(slice(0, B)), zip(*parts)))


@pytest.mark.parametrize("D,dtype,Hq,Hkv", [(128, BF, 6, 2), (64, HF, 5, 1)])
@pytest.mark.parametrize("n", [1216, 1217, 2432, 3648, 3649, 3651])
def test_packed_tokens(D, dtype, Hq, Hkv, n):
    r, ps, rng = turning(D), 32, np.random.default_rng(n)
    q, k, v = rows(dtype, n, Hq, D), rows(dtype, n, Hkv, D), rows(dtype, n, Hkv, D)
    cut = np.sort(rng.integers(0, n - 3, 5))
    cu = np.concatenate([[0], cut, [n - 3]])                     # (three rows behind the last sequence)
    new = np.diff(cu)
    lens = new + rng.integers(0, 100, 6)
    width = int(-(-lens.max() // ps))
    table = rng.permutation(6 * width).reshape(6, width)

    def caches():
        return [torch.full((1, 6 * width, ps, Hkv, D), 7.0, dtype=dtype, device="cuda") for _ in range(2)]

    def call(first, last, kc, vc):
        at = slice(int(cu[first]), n if last == 6 else int(cu[last]))
        d = kv.make_kv_dims(last - first, 1, Hq, Hkv, D, ps, 6 * width, width, 6, first, dtype=dtype)
        q_out = torch.full_like(q[at], 7.0)
        kv.gdn_kv_append(d, 0, r, i32(cu[first:last + 1] - cu[first]), q[at], k[at], v[at], None, kc, vc, i32(table), i32(lens), None, q_out)
        return q_out

    whole, pieces = caches(), caches()
    q_out = call(0, 6, *whole)
    assert (q_out[n - 3:] == 7.0).all()
    assert torch.equal(q_out, torch.cat([call(b, b + 1, *pieces) for b in range(6)]))
    assert all(torch.equal(a, b) for a, b in zip(whole, pieces)) and not (whole[0] == 7.0).all()
