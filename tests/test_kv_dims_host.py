"""Dims of the paged cache's calls from tensors whose single entries have strides of their own."""
import ctypes

import pytest

from test_kv_host import BASE, BIG, attn, commit, lib, ptrs  # noqa: F401

from speculative_decode_verify_gdn_gb300 import gdn, kv

torch = pytest.importorskip("torch")


def test_one_token_has_no_step_to_the_next(lib):
    """A single token [1, 1, heads, D] cut from [heads, 1, D] has the stride of a head between its
    tokens; nothing steps over it."""
    one = dict(BASE, B=1, K=1)
    q = torch.empty(1, 4, 1, 64).transpose(1, 2).as_strided((1, 1, 4, 64), (64, 64, 64, 1))
    w = torch.empty(2, 2, 1, 64).transpose(1, 2).unsqueeze(1).as_strided((2, 1, 1, 2, 64), (128, 64, 64, 64, 1))
    d = kv.make_kv_dims(**one, q=q, win=w)
    assert d.q_token_stride >= 4 * 64 and d.win_token_stride >= 2 * 64 and d.win_layer_stride == 128
    for call, n in ((attn, 13), (commit, 13)):
        a = ptrs(n)
        a[12] = a[11]                # all but the last of the checks pass
        assert call(lib, d, a) == gdn.GDN_ERR_ALIAS
    d = kv.make_kv_dims(**dict(one, n_layers=1), win=w[0])
    assert d.win_token_stride >= 2 * 64


def test_steps_between_sequences_of_one_token_and_between_tokens(lib):
    qkv = torch.empty(3, 1, 9 * 64)
    d = kv.make_kv_dims(**dict(BASE, B=3, K=1, n_slots=3), q=qkv[..., :256].view(3, 1, 4, 64),
                        win=qkv[..., 256:384].view(3, 1, 2, 64))
    assert d.q_token_stride == 576 and d.win_token_stride == 576
    d = kv.make_kv_dims(**dict(BASE, B=1, K=3), q=qkv.view(1, 3, 576)[..., :256].view(1, 3, 4, 64),
                        win=qkv.view(1, 3, 576)[..., 256:384].view(1, 3, 2, 64))
    assert d.q_token_stride == 576 and d.win_token_stride == 576
