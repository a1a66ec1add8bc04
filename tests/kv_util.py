"""Inputs of the paged key/value cache tests: a pool in which everything that no call may read is
NaN, as CUDA tensors and as the float64 arrays the oracle takes."""
import numpy as np
import torch

from speculative_decode_verify_gdn_gb300 import kv

# Bits of relative rounding error of the 16-bit types: at most 2^-8 for bf16, 2^-11 for f16.
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def f64(t):
    return t.double().cpu().numpy()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Pool:
    """lens[s] tokens in slot s, on pages scattered over the pool; order 'nhd' or 'hnd' (of a page),
    or 'mixed': keys and values of a page next to each other in one tensor."""

    def __init__(self, seed, lens, *, ps=16, Hkv=2, D=64, layers=1, dtype=torch.bfloat16, order="nhd", n_pages=None,
                 max_pages=None, spare=3):
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.lens = np.asarray(lens, dtype=np.int64)
        self.ps, self.Hkv, self.D, self.layers, self.dtype = ps, Hkv, D, layers, dtype
        pages = -(-self.lens // ps)
        self.n_pages = int(pages.sum()) + spare if n_pages is None else n_pages
        self.max_pages = max(1, int(pages.max(initial=0)) + 1) if max_pages is None else max_pages
        ids = self.rng.permutation(self.n_pages)
        self.table = np.full((len(lens), self.max_pages), -1, dtype=np.int64)
        self.ref = np.zeros(self.n_pages, dtype=np.int64)
        at = 0
        for s, n in enumerate(pages):
            self.table[s, :n] = ids[at:at + n]
            self.ref[ids[at:at + n]] += 1
            at += n
        L, P = layers, self.n_pages
        if order == "nhd":
            self.k, self.v = (self.nan((L, P, ps, Hkv, D)) for _ in range(2))
        elif order == "hnd":
            self.k, self.v = (self.nan((L, P, Hkv, ps, D)).transpose(2, 3) for _ in range(2))
        else:
            both = self.nan((L, P, 2, ps, Hkv, D))
            self.k, self.v = both[:, :, 0], both[:, :, 1]
        for s, n in enumerate(self.lens):
            for c in range(int(pages[s])):
                fill = min(ps, int(n) - c * ps)
                for x in (self.k, self.v):
                    x[:, self.table[s, c], :fill] = self.gauss((L, fill, Hkv, D))

    def nan(self, shape):
        return torch.full(shape, float("nan"), dtype=self.dtype, device="cuda")

    def gauss(self, shape, scale=1.0):
        t = torch.empty(shape, dtype=self.dtype, device="cuda")
        return t.normal_(0.0, scale, generator=self.gen)

    def dims(self, B=0, K=1, Hq=None, slot0=0, q=None, win=None):
        return kv.make_kv_dims(B, K, Hq or self.Hkv, self.Hkv, self.D, self.ps, self.n_pages, self.max_pages,
                               len(self.lens), slot0, self.layers, self.dtype, cache=self.k, q=q, win=win)


def random_trees(rng, B, K):
    return np.stack([[int(rng.integers(-1, t)) if t and rng.random() < 0.5 else t - 1 for t in range(K)]
                     for _ in range(B)])
