"""The paged cache in use: the hybrid round of examples/hybrid_round.py against the oracle, and the
cache's in-place round against the out-of-place calls."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from kv_util import ROUND, f64
from oracle import kv_oracle as O
from speculative_decode_verify_gdn_gb300 import gdn, kv
from speculative_decode_verify_gdn_gb300.build import build_library

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    build_library()
    kv.load_library()
    gdn.gdn_device_status(clear=True)
    yield
    assert gdn.gdn_device_status(clear=True) == 0


def example():
    spec = importlib.util.spec_from_file_location("hybrid_round", os.path.join(ROOT, "examples", "hybrid_round.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_hybrid_round_example():
    """Every round's attention output is the oracle's on what the cache held then (the tolerance of
    test_gpu_kv_attn.py), and the books balance at the end."""
    m = example()
    B, K, D = 4, 5, 64
    cache, state, seen = m.run(B=B, K=K, prompt=77, rounds=5, seed=3)
    assert torch.isfinite(state.state).all()
    for r in seen:
        table, lens = r["table"].cpu().numpy(), r["lens"].cpu().numpy()
        for layer in range(m.LAYERS):
            q, kw, vw = (f64(r[x][layer]) for x in ("q", "k_win", "v_win"))
            k, v = np.nan_to_num(f64(r["k"][layer])), np.nan_to_num(f64(r["v"][layer]))
            args = (table, lens, [B] * B, None, None, D ** -0.5)
            ref, _ = O.attention(q, kw, vw, k, v, *args)
            mag, _ = O.attention(q, kw, np.abs(vw), k, np.abs(v), *args)
            assert (np.abs(f64(r["out"][layer]) - ref) <= ROUND[torch.bfloat16] * (mag + np.abs(ref)) + 2e-4 * mag).all()
    lens, table, ref = (x.cpu().numpy() for x in (cache.seq_len, cache.table, cache.ref))
    count = np.zeros_like(ref)
    for s, n in enumerate(lens):
        np.add.at(count, table[s, :-(-int(n) // cache.page_size)], 1)
    assert np.array_equal(count, ref)
    live = int(cache.n_live)
    assert (ref[:live] > 0).all() and (ref[live:] == 0).all()


def test_example_command(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["hybrid_round.py", "--rounds", "3"])
    example().main()
    assert "3 rounds" in capsys.readouterr().out


def test_window_commit_equals_what_attention_saw():
    """Attention over a window equals attention of its last token once the rest is committed."""
    m = example()
    cache, _, _ = m.run(B=3, K=4, prompt=50, rounds=1, seed=5)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    q, kw, vw = (torch.empty((2, 3, 4, h, 64), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for h in (8, 2, 2))
    out = torch.empty_like(q[0])
    cache.attend(1, q[1], kw[1], vw[1], out)
    cache.commit(torch.full((3,), 3, dtype=torch.int32, device="cuda"), kw, vw)
    last = torch.empty_like(out)
    # the fourth token alone is this round's window: the first of its four, the others padding
    q1, k1, v1 = (torch.roll(x[1], -3, dims=1).contiguous() for x in (q, kw, vw))
    cache.attend(1, q1, k1, v1, last, win_len=torch.ones(3, dtype=torch.int32, device="cuda"))
    # the same keys in other tiles: rounding of the probabilities alone, twice 2^-8 of values up to 4
    assert (last[:, 0].float() - out[:, 3].float()).abs().max() <= 2 * 2.0 ** -8 * vw.abs().max().float() * 2
