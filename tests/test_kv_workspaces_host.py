"""Whose scratch PagedCache's attentions run in, with the library's calls and the streams replaced."""
import contextlib
import types

import pytest

from speculative_decode_verify_gdn_gb300 import build, gdn, kv
from speculative_decode_verify_gdn_gb300.kv_runtime import PagedCache

torch = pytest.importorskip("torch")


@pytest.fixture
def world(monkeypatch):
    """Streams by name, the current one last, and those that are being captured."""
    build.build_library()
    w = types.SimpleNamespace(current=["main"], captured=set(), made=[], used=[])

    @contextlib.contextmanager
    def stream(s):
        w.current.append(w.current[-1] if s is None else s.cuda_stream)
        yield
        w.current.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: w.current[-1] in w.captured)
    monkeypatch.setattr(kv, "_capturing", lambda s: s.cuda_stream in w.captured)
    monkeypatch.setattr(kv, "_current_device", lambda: 0)
    monkeypatch.setattr(kv, "_current_stream", lambda device: w.current[-1])
    for name in ("alloc_attn_workspace", "alloc_attn_prefill_workspace"):
        def made(*args, f=getattr(kv, name), name=name):
            w.made.append((name, w.current[-1]))
            return f(*args)
        made.__name__ = name
        monkeypatch.setattr(kv, name, made)
    monkeypatch.setattr(kv, "gdn_attn_verify", lambda *args: w.used.append(args[-2]))
    monkeypatch.setattr(kv, "gdn_attn_prefill", lambda *args: w.used.append(args[-2]))
    return w


def named(s):
    return None if s is None else types.SimpleNamespace(cuda_stream=s)


def test_a_workspace_for_each_stream_and_each_capture(world):
    c = PagedCache.create(2, 1, 2, 1, 64, 16, n_pages=20, max_pages=4, device="cpu")
    c.k = types.SimpleNamespace(is_cuda=True, device="cpu")
    rows, cu = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)

    def calls(s):
        c.attend(0, rows, None, None, rows, stream=named(s))
        c.attend_prefill(0, cu, rows, rows, stream=named(s))
        return world.used[-2:]

    assert world.made == []                                     # (a cache that is never attended has none)
    main, side, third = calls(None), calls("side"), calls("third")
    assert [m for _, m in world.made] == ["main", "main", "side", "side", "third", "third"]
    for again, first in ((calls(None), main), (calls("main"), main), (calls("side"), side), (calls("third"), third)):
        assert all(a is b for a, b in zip(again, first))
    assert len({t.data_ptr() for t in main + side + third}) == 6 and len(world.made) == 6
    world.captured.add("side")                                  # two graphs, captured one after the other on one stream
    graphs = [calls("side") for _ in range(2)]
    assert [m for _, m in world.made[6:]] == ["side"] * 4
    assert len({t.data_ptr() for t in graphs[0] + graphs[1] + side}) == 6
    assert all(a is b for a, b in zip(calls("third"), third))   # (not a part of the capture)
    world.captured.clear()
    assert all(a is b for a, b in zip(calls("side"), side))
    world.current[:] = ["side"]
    assert all(a is b for a, b in zip(calls(None), side))
    for t, size in zip(main, (kv.gdn_attn_workspace_size(c.dims), kv.gdn_attn_prefill_workspace_size(c.dims, 1000))):
        assert t.numel() >= size


@pytest.mark.parametrize("B,n_prefixes", [(65535, 0), (65535, 1), (3, 65533), (1000, 70000)])
def test_the_pool_has_room_for_the_largest_call(B, n_prefixes):
    """More slots than a call may name sequences: the workspace serves a commit of all B and a reserve of as many slots as
    a call takes."""
    build.build_library()
    c = PagedCache.create(B, 1, 1, 1, 64, 16, n_pages=4, max_pages=1, n_prefixes=n_prefixes, device="cpu")
    assert c.pool_workspace.numel() >= kv.gdn_kv_workspace_size(c.dims)
    assert c.pool_workspace.numel() >= kv.gdn_kv_workspace_size(c._dims(min(65535, B + n_prefixes)))
    assert kv.gdn_kv_workspace_size(c._dims(65535 if B + n_prefixes > 65535 else 1)) > kv.gdn_kv_workspace_size(c._dims(0))


@pytest.mark.parametrize("over", [dict(K=17), dict(B=65536), dict(Hq=3, Hkv=2), dict(D=96), dict(page_size=24), dict(Hq=129)])
def test_a_cache_that_no_attention_takes_is_refused_at_once(over):
    build.build_library()
    args = dict(B=2, K=1, Hq=1, Hkv=1, D=64, page_size=16, n_pages=4, max_pages=1, device="cpu")
    with pytest.raises(gdn.GdnError):
        PagedCache.create(**dict(args, **over))
