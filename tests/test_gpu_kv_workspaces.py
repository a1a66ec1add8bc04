"""Attention of one cache on several streams at once, and in graphs that were captured on one stream and are replayed on
two: the same bits as one after the other."""
import pytest
import torch

from kv_util import i32
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


def rows(*shape):
    return torch.empty(shape, dtype=BF, device="cuda").normal_()


@pytest.fixture(scope="module")
def cache():
    """Long slots, so that every call below is cut into pieces that go through the workspace."""
    c = PagedCache.create(4, 4, 8, 2, 128, 64, n_pages=1000, max_pages=250)
    for slot, n in enumerate((9000, 15000, 30, 12000)):
        c.append(slot, rows(1, n, 2, 128), rows(1, n, 2, 128))
    return c


def prefill(c, slot0, new, q, out, lse):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    bounds = i32(cu)
    torch.cuda.synchronize()
    return lambda stream=None: c.attend_prefill(0, bounds, q, out, lse, slot0, stream=stream)


def jobs(c, attend):
    """Calls and their outputs: prefill attention of different sequences (few rows, and tiles), or the windows'."""
    made = []
    for slot0, new in ((0, [300, 1]), (1, [1, 1, 1]), (3, [40]), (0, [1, 700, 0, 5])):
        if attend:
            q, k, v = rows(4, 4, 8, 128), rows(4, 4, 2, 128), rows(4, 4, 2, 128)
            out, lse = torch.empty_like(q), torch.empty((4, 4, 8), device="cuda")
            made.append((lambda stream=None, a=(q, k, v, out, lse): c.attend(0, *a, stream=stream), (out, lse)))
        else:
            q = rows(sum(new), 8, 128)
            out, lse = torch.empty_like(q), torch.empty((sum(new), 8), device="cuda")
            made.append((prefill(c, slot0, new, q, out, lse), (out, lse)))
    return made


def copies(made):
    return [t.clone() for _, outs in made for t in outs]


@pytest.mark.parametrize("attend", [False, True])
def test_streams_at_once(cache, attend):
    made = jobs(cache, attend)
    for call, _ in made:
        call()
    want = copies(made)
    streams = [torch.cuda.Stream() for _ in made]
    for _, outs in made:
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for (call, _), s in zip(made, streams):
            call(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, copies(made)))


def test_whether_a_stream_is_captured():
    """The capture's stream and one that joined it, but none beside; the current stream stays what it was."""
    main, side, other = torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()
    x = torch.zeros(4, device="cuda")

    def look():
        before = torch.cuda.current_stream()
        seen = [kv.stream_state(s) for s in (None, side, other)]
        assert torch.cuda.current_stream() == before
        assert [h for h, _ in seen] == [before.cuda_stream, side.cuda_stream, other.cuda_stream]
        return [c for _, c in seen]

    assert look() == [False, False, False]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1)
        assert look() == [True, False, False]
        side.wait_stream(torch.cuda.current_stream())
        assert look() == [True, True, False]
        torch.cuda.current_stream().wait_stream(side)
    assert look() == [False, False, False] and torch.cuda.current_stream() == main


@pytest.mark.parametrize("attend", [False, True])
def test_graphs_at_once(cache, attend):
    made = jobs(cache, attend)
    for call, _ in made:
        call()
    want = copies(made)
    torch.cuda.synchronize()
    graphs = []
    for call, _ in made:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
            call()
    streams = [torch.cuda.Stream() for _ in made]
    for _, outs in made:
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for (call, _) in made[:1]:  # (and an eager call beside them, of outputs that a graph writes the same bits to)
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, copies(made)))
