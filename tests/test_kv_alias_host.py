"""Which placements of the key and the value cache the calls that write them accept: interleaved in
one buffer, but with no element in common.  Every call here fails validation before the library
touches CUDA: no GPU is needed and no kernel is launched."""
import ctypes
import itertools

import pytest

from speculative_decode_verify_gdn_gb300 import build, gdn, kv

torch = pytest.importorskip("torch")
MB = 1 << 24
P = 1 << 40          # never dereferenced
BIG = ctypes.c_uint64(1 << 40)


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return kv.load_library()


def calls(lib, d, k, v):
    """What commit, fork and compact say of these cache addresses.  The workspace lies over the output
    before it, which is looked at last: an accepted placement ends there."""
    out = []
    for f, n, at in ((lib.gdn_kv_commit, 13, 4), (lib.gdn_kv_fork, 10, 1), (lib.gdn_kv_compact, 9, 0)):
        a = [P + (i + 1) * 64 * MB for i in range(n)]
        a[at], a[at + 1] = k, v
        a[-1] = a[-2]
        status = f(ctypes.byref(d), *a, BIG, None)
        assert status == gdn.GDN_ERR_ALIAS
        out.append(gdn.last_error())
    return out


def accepted(lib, d, k, v):
    got = ["workspace" in text for text in calls(lib, d, k, v)]
    assert len(set(got)) == 1
    return got[0]


def dims(layers=2, pages=3, ps=16, Hkv=2, D=64, strides=None):
    d = kv.make_kv_dims(2, 4, 4, Hkv, D, ps, pages, 4, n_slots=3, n_layers=layers)
    if strides:
        d.cache_layer_stride, d.cache_page_stride, d.cache_token_stride, d.cache_head_stride = strides
    return d


def test_dense_caches_may_not_overlap(lib):
    d = dims()
    size = 2 * 2 * 3 * 16 * 2 * 64
    for off in (16, 128, 256, 2 * 16 * 2 * 64, 3 * 2 * 16 * 2 * 64, size - 16):   # up to whole pages and layers
        assert not accepted(lib, d, P, P + off) and not accepted(lib, d, P + off, P), off
    assert accepted(lib, d, P, P + size) and accepted(lib, d, P + size, P)


def test_keys_and_values_in_one_buffer(lib):
    L, N, ps, H, D = 2, 3, 16, 2, 64
    row, page = H * D, ps * H * D
    for strides, off in (
            ((2 * N * page, 2 * page, row, D), page),              # [L, N, 2, ps, H, D]
            ((2 * N * page, 2 * page, D, ps * D), page),           # [L, N, 2, H, ps, D]
            ((2 * N * page, page, row, D), N * page),              # [L, 2, N, ps, H, D]
            ((2 * N * page, 2 * page, 2 * row, D), row),           # [L, N, ps, 2, H, D]
            ((2 * N * page, 2 * page, 2 * row, 2 * D), D),         # [L, N, ps, H, 2, D]
            ((2 * N * page, 2 * page, row, D), 3 * page)):         # values one page further on
        d = dims(L, N, ps, H, D, strides)
        assert accepted(lib, d, P, P + 2 * off) and accepted(lib, d, P + 2 * off, P), strides
        assert not accepted(lib, d, P, P + 2 * off + 16), strides


def test_every_placement_against_the_elements(lib):
    """Small strided caches at every distance of 8 elements: accepted exactly where no element is shared."""
    L, N, ps, H, D = 2, 2, 16, 2, 64
    row, page = H * D, ps * H * D
    for strides in ((N * page, page, row, D), (2 * N * page, 2 * page, row, D), (2 * N * page, 2 * page, 2 * row, D + 8),
                    (D * H * ps + 16, 2 * (D * H * ps + 16), D, D * ps)):
        d = dims(L, N, ps, H, D, strides)
        rows = {sum(i * s for i, s in zip(at, strides)) for at in itertools.product(range(L), range(N), range(ps), range(H))}
        starts = {r + 8 * e for r in rows for e in range(D // 8)}
        extent = max(starts) + 8
        for off in list(range(8, extent, 8 * 37)) + [r for r in sorted(rows) if r][:40] + [extent - 8, extent]:
            shared = any(s + off in starts for s in starts)
            assert accepted(lib, d, P, P + 2 * off) == (not shared), (strides, off)
