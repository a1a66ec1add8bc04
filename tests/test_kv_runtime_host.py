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
