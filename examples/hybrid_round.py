"""Speculative-decoding rounds of a small hybrid model: one GDN layer and two softmax-attention
layers over random activations (no weights: the layers' inputs are drawn, as in synth.py).

    python examples/hybrid_round.py [--rounds N]

A prompt shared by all sequences is prefilled once - its GDN state is copied to every sequence,
its keys and values go to pages that all of them read.  Each round drafts a window of K tokens per
sequence, verifies it in the GDN layer (chain) and the attention layers, and keeps the accepted
tokens: the GDN state is rolled back, the window's keys and values are committed to pages.  Half
way the sequences are resampled (forked and dropped), and at the end the pool is compacted.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decode_verify_gdn_gb300 import gdn  # noqa: E402
from speculative_decode_verify_gdn_gb300.kv_runtime import PagedCache  # noqa: E402
from speculative_decode_verify_gdn_gb300.runtime import GdnLayerState  # noqa: E402
from speculative_decode_verify_gdn_gb300.synth import Dims, Dists, Gen, make_layer, make_prompts, make_round  # noqa: E402

LAYERS = 2


def run(B=6, K=8, prompt=300, rounds=6, Hq=8, Hkv=2, D=64, page_size=16, seed=0, device="cuda:0"):
    """Returns the cache, the GDN layer's state, and each round's attention outputs with their inputs."""
    torch.cuda.set_device(device)
    g = Gen(seed)
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    d = Dims(B=B, K=K, Hk=2, Hv=4, dk=64, dv=64)

    def gauss(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=device).normal_(0.0, 1.0, generator=gen)

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)

    # the prompt: GDN prefill of one sequence, its state copied to all; keys and values to slot B
    layer = make_layer(g, d, Dists())
    state = GdnLayerState.create(d, layer, device=device, keep_snapshot=True, out_f32=False)
    one = Dims(B=1, K=1, Hk=d.Hk, Hv=d.Hv, dk=d.dk, dv=d.dv)
    drawn = make_prompts(g, one, [prompt], Dists())
    dims = gdn.make_dims(1, 1, one.Hk, one.Hv, one.dk, one.dv, one.W, 1.0, 1e-6, 0)
    x, a, b = (torch.from_numpy(np.ascontiguousarray(t).view(np.int16)).to(device).view(torch.bfloat16)
               for t in (drawn.x, drawn.a, drawn.b))
    S, CS = torch.zeros_like(state.state[:1]), torch.zeros_like(state.conv_state[:1])
    gdn.gdn_prefill(dims, ints([0, prompt]), x, a, b, state.A_log, state.dt_bias, state.conv_w, CS, CS, S, S,
                    torch.empty((prompt, d.Hv, d.dv), dtype=torch.bfloat16, device=device),
                    gdn.alloc_prefill_workspace(dims, prompt, device))
    state.state.copy_(S.expand_as(state.state))
    state.conv_state.copy_(CS.expand_as(state.conv_state))

    longest = prompt + rounds * K
    cache = PagedCache.create(B, K, Hq, Hkv, D, page_size, n_pages=-(-prompt // page_size) + 2 * B * (rounds * K // page_size + 2),
                              max_pages=-(-longest // page_size), n_prefixes=1, n_layers=LAYERS, device=device)
    cache.append(B, gauss(LAYERS, prompt, Hkv, D), gauss(LAYERS, prompt, Hkv, D))
    cache.prefix_of.fill_(B)

    seen = []
    for r in range(rounds):
        state.load_round(make_round(g, d, Dists()))
        accept = ints(rng.integers(1, K + 1, B))
        state.accept_len.copy_(accept)
        state.verify()
        q, k_win, v_win = gauss(LAYERS, B, K, Hq, D), gauss(LAYERS, B, K, Hkv, D), gauss(LAYERS, B, K, Hkv, D)
        out = torch.empty_like(q)
        for layer_index in range(LAYERS):
            cache.attend(layer_index, q[layer_index], k_win[layer_index], v_win[layer_index], out[layer_index])
        seen.append(dict(q=q, k_win=k_win, v_win=v_win, out=out, table=cache.table.clone(), lens=cache.seq_len.clone(),
                         k=cache.k.clone(), v=cache.v.clone()))
        state.rollback()
        cache.commit(accept, k_win, v_win)
        if r == rounds // 2:  # resample: the cache forks, the GDN states are gathered
            src = np.sort(rng.integers(0, B, B))
            cache.fork(ints(np.append(src, B)))
            at = torch.from_numpy(src).to(device)
            state.state.copy_(state.state[at])
            state.conv_state.copy_(state.conv_state[at])
    cache.compact()
    return cache, state, seen


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rounds", type=int, default=6)
    args = ap.parse_args()
    cache, state, seen = run(rounds=args.rounds)
    torch.cuda.synchronize()
    flags = gdn.gdn_device_status()
    if flags:
        raise SystemExit(f"device status {flags:#x}")
    print(f"{len(seen)} rounds, sequence lengths {cache.seq_len[:cache.B].tolist()} behind a prompt of "
          f"{int(cache.seq_len[cache.B])} tokens, {int(cache.n_live)} of {cache.n_pages} pages in use, "
          f"GDN state norm {state.state.norm().item():.4g}")


if __name__ == "__main__":
    main()
