"""Host side of the paged cache's runtime, with the library's calls replaced: which stream a method's
own memory and work belong to, and what it passes on."""
import contextlib

import pytest

from speculative_decode_verify_gdn_gb300 import build, kv
from speculative_decode_verify_gdn_gb300.kv_runtime import PagedCache

torch = pytest.importorskip("torch")


class FakeStream:
    cuda_stream = 7


@pytest.fixture
def on(monkeypatch):
    """The streams that are current, innermost last, as torch.cuda.stream sets them."""
    build.build_library()
    streams = [None]

    @contextlib.contextmanager
    def stream(s):
        streams.append(streams[-1] if s is None else s)
        yield
        streams.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    return streams


def cache(B=3, n_prefixes=2, **over):
    args = dict(K=4, Hq=4, Hkv=2, D=64, page_size=16, n_pages=20, max_pages=4, n_layers=2, device="cpu")
    return PagedCache.create(B, n_prefixes=n_prefixes, **dict(args, **over))


def test_append_allocates_and_fills_on_the_stream_it_runs_on(on, monkeypatch):
    """The accept length and the workspace belong to the commit's stream: filled in its order, and
    not handed to other work while it runs."""
    made, calls = [], []

    def seen(f):
        def g(*args, **kw):
            made.append(on[-1])
            return f(*args, **kw)
        return g

    c = cache()
    monkeypatch.setattr(torch, "full", seen(torch.full))
    monkeypatch.setattr(kv, "alloc_kv_workspace", seen(kv.alloc_kv_workspace))
    monkeypatch.setattr(kv, "gdn_kv_commit", lambda *args: calls.append((args[1], args[-1])))
    new = torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)
    side = FakeStream()
    for stream in (side, None):
        made.clear()
        c.append(1, new, new, stream=stream)
        assert made and all(m is stream for m in made)
        accept, passed = calls[-1]
        assert passed is stream and accept.tolist() == [5]


def test_fork_takes_the_prefix_along(on, monkeypatch):
    """Sequence i goes on behind the prefix of the sequence it takes.  One that goes on from a prefix's own
    slot has none behind it; a dropped slot, or one whose source is no slot, keeps its entry."""
    seen = []
    monkeypatch.setattr(kv, "gdn_kv_fork", lambda *args: seen.append((on[-1], args[-1])))
    c = cache(B=5)
    prefix_of = c.prefix_of
    side = FakeStream()
    for src, before, after in (([1, 0, 3, 3, -1, 5, 6], [5, 6, -1, 6, 5], [6, 5, 6, 6, 5]),
                               ([4, 4, 2, 2, 0, 5, 6], [5, 6, -1, 6, 6], [6, 6, -1, -1, 5]),
                               ([5, 6, -9, 7, 1, 5, 6], [5, 5, 6, 5, 6], [-1, -1, 6, 5, 5])):
        prefix_of.copy_(torch.tensor(before, dtype=torch.int32))
        c.fork(torch.tensor(src, dtype=torch.int32), stream=side)
        assert c.prefix_of is prefix_of and prefix_of.tolist() == after
    assert seen[-1][1] is side
    alone = cache(n_prefixes=0)
    alone.fork(torch.tensor([2, 1, 0], dtype=torch.int32))
    assert alone.prefix_of.tolist() == [-1, -1, -1] and seen[-1][1] is None
