"""Workspace sizes of the paged cache's calls.  Every call here fails validation before the library
touches CUDA: no GPU is needed and no kernel is launched."""
import ctypes

from test_kv_host import INV, commit, compact, dims, fork, lib, ptrs, with_field  # noqa: F401

from speculative_decode_verify_gdn_gb300 import gdn, kv


def test_fork_and_compact_do_not_read_the_batch(lib):
    """A workspace sized for a pool with no batch serves fork and compact whatever B says; sizes for a
    commit grow with B, and a B that commit refuses asks for no more than none."""
    pool = dims(B=0)
    size = kv.gdn_kv_workspace_size(pool)
    assert kv.gdn_kv_workspace_size(dims(B=2)) <= kv.gdn_kv_workspace_size(with_field("B", 65535, n_slots=3))
    for b in (0, 2, 65535, 65536, (1 << 31) - 1, -1):
        d = with_field("B", b)
        if b < 0 or b > 65535:
            assert kv.gdn_kv_workspace_size(d) == size
        for call, n in ((fork, 10), (compact, 9)):
            a = ptrs(n)
            a[-1] = a[-2]            # the last of the checks: the workspace over the output before it
            assert call(lib, d, a, ctypes.c_uint64(size)) == gdn.GDN_ERR_ALIAS, b
            assert call(lib, d, a, ctypes.c_uint64(16)) == INV and "workspace" in gdn.last_error()
    d = dims(B=2, n_slots=300)
    d.B = 300
    assert commit(lib, d, ws=ctypes.c_uint64(kv.gdn_kv_workspace_size(dims(B=1, n_slots=300)))) == INV
    assert "workspace" in gdn.last_error()
