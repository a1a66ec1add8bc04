"""Host side of what reserve notes about the sequences that it had no room for: arguments of the calls that
write and read it, and what PagedCache passes on.  No kernel is launched."""
import ctypes

import pytest

from speculative_decode_verify_gdn_gb300 import build, gdn, kv
from speculative_decode_verify_gdn_gb300.kv_runtime import PagedCache
from test_kv_prompt_host import BIG, N, ptrs, dims, ref, turning

torch = pytest.importorskip("torch")
INV, ALIAS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_ALIAS


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return kv.load_library()


# n_new table_in table_out len_in len_out ref_in ref_out refused workspace
def reserve(lib, a):
    return lib.gdn_kv_reserve_marked(ref(dims()), *a, BIG, None)


# turns q_weight k_weight | cu q k v positions k_cache v_cache table seq_len refused prefix_of q_out
def append(lib, a):
    return lib.gdn_kv_append_marked(ref(dims()), 0, ref(turning()), *a[:3], N, *a[3:], None)


# cu q k_cache v_cache table seq_len refused prefix_of | out lse workspace
def prefill(lib, a):
    return lib.gdn_attn_prefill_marked(ref(dims()), 0, N, *a[:8], 1, 0.125, *a[8:], BIG, None)


@pytest.mark.parametrize("call,n,refused,others", [
    (reserve, 9, 7, range(9)), (append, 15, 12, (8, 9, 14)), (prefill, 11, 6, (8, 9, 10))])
def test_arguments(lib, call, n, refused, others):
    """refused is aligned like other int32 arrays, and shares no element with an output."""
    a = ptrs(n)
    a[refused] += 2
    assert call(lib, a) == INV and "refused is not" in gdn.last_error()
    for i in others:
        if i != refused:
            a = ptrs(n)
            a[refused] = a[i]
            assert call(lib, a) == ALIAS and "refused" in gdn.last_error(), i


def test_the_cache_passes_it_on(monkeypatch):
    """Reserve writes the cache's entries, append and prefill attention read the same; a fork, whose slots hold other
    sequences behind it, takes them back."""
    build.build_library()
    calls = []
    for name, at in (("gdn_kv_reserve", 5), ("gdn_kv_append", 11), ("gdn_attn_prefill", 7)):
        monkeypatch.setattr(kv, name, lambda *args, at=at: calls.append(args[at]))
    monkeypatch.setattr(kv, "gdn_kv_fork", lambda *args: None)
    c = PagedCache.create(3, 1, 2, 1, 64, 16, n_pages=20, max_pages=4, n_prefixes=1, device="cpu")
    assert c.refused.dtype is torch.int32 and c.refused.tolist() == [-1] * 4
    rows, cu = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    for _ in range(2):
        calls.clear()
        c.reserve(torch.zeros(3, dtype=torch.int32))
        c.append_layer(0, None, cu, rows, rows[:, :1], rows[:, :1], rows)
        c.attend_prefill(0, cu, rows, torch.empty_like(rows))
        assert len(calls) == 3 and all(lens is c.seq_len and noted is c.refused for lens, noted in calls)
        c.refused.fill_(7)
        c.fork(torch.arange(4, dtype=torch.int32))
        assert c.refused.tolist() == [-1] * 4


def test_the_binding_takes_a_pair():
    t = torch.zeros(3, dtype=torch.int32)
    assert kv._lengths(t, "seq_len", 3, -1) == (t.data_ptr(), None)
    u = t.clone()
    assert kv._lengths((t, u), "seq_len", 3, -1) == (t.data_ptr(), u.data_ptr())
    for bad in ((t, u[:2]), (t, u.long()), (u[:2], t)):
        with pytest.raises((TypeError, ValueError)):
            kv._lengths(bad, "seq_len", 3, -1)
    assert ctypes.sizeof(kv.KvDims) and "gdn_kv_append_marked" in kv.EXPORTED
