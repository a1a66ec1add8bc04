"""Cases of the operators that bring prompts into the paged key/value cache and a verify window's queries and keys
into place: norms and rotation of a window, pages for new tokens, append of ragged tokens of one layer, and the
attention of ragged queries over the cache (causal, or to an encoder's states).

    listed()              the named cases
    draw(rng)             one more case of the same ranges
    prepare(case, seed)   inputs on the GPU
    run(state)            one pass: in plain torch operations, or (own) through the library
    exact(case, seed)     the same outputs from the definition in 64 bits
    work(case)            bytes and operations the pass cannot do without
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # plain decode of one user: the latency end; queries with a gate beside each head's
        dict(name="rope one decode token", op="rope", B=1, K=1, Hq=16, Hkv=2, D=128, dtype="bf16", P=0, plen=0, lo=700,
             hi=700, tree=False, ragged=False, rot=32, inter=False, norm=True, stretch=1.0, gate=True),
        # a serving batch of drafted trees, padded windows, far positions on frequencies stretched for long contexts
        dict(name="rope serving trees", op="rope", B=256, K=16, Hq=32, Hkv=8, D=128, dtype="bf16", P=1, plen=120000,
             lo=1, hi=4096, tree=True, ragged=True, rot=128, inter=False, norm=True, stretch=4.0, gate=False),
        # plain decode of 32 users in one layer: a token each
        dict(name="append a token each", op="append", B=32, Hq=32, Hkv=8, D=128, ps=64, dtype="bf16", P=1, plen=1000,
             nlo=1, nhi=1, lo=5, hi=1024, rot=128, inter=False, norm=True, stretch=1.0, gate=False),
        # a batch of prompts of one layer, some of them continued ones
        dict(name="append ragged prompts", op="append", B=9, Hq=32, Hkv=8, D=128, ps=64, dtype="bf16", P=0, plen=0,
             nlo=1, nhi=8191, lo=0, hi=700, rot=128, inter=False, norm=True, stretch=1.0, gate=False),
        # one user's next token
        dict(name="reserve for one sequence", op="reserve", B=1, ps=16, n_pages=256, nlo=4, nhi=4, lo=700, hi=700),
        # a full pool, prompts of many users arriving
        dict(name="reserve for many prompts", op="reserve", B=256, ps=16, n_pages=40000, nlo=0, nhi=600, lo=1, hi=1500),
        # one short prompt of one user: latency
        dict(name="prefill a short prompt", op="attn", B=1, Hq=16, Hkv=2, D=128, ps=16, dtype="bf16", P=0, plen=0,
             nlo=37, nhi=37, lo=0, hi=0, causal=True),
        # questions of 13 users behind one system prompt, f16, small heads, pages of 48 tokens
        dict(name="prefill ragged prompts", op="attn", B=13, Hq=24, Hkv=4, D=64, ps=48, dtype="f16", P=1, plen=1531,
             nlo=1, nhi=901, lo=0, hi=333, causal=True),
        # the next chunk of a long prompt: few rows, a long axis
        dict(name="prefill a late chunk", op="attn", B=1, Hq=32, Hkv=8, D=128, ps=64, dtype="bf16", P=0, plen=0,
             nlo=512, nhi=512, lo=65536, hi=65536, causal=True),
        # long prompts of several users: the matrix-product end
        dict(name="prefill long prompts", op="attn", B=4, Hq=32, Hkv=8, D=128, ps=64, dtype="bf16", P=0, plen=0,
             nlo=4096, nhi=16384, lo=0, hi=0, causal=True),
        # decode of an encoder-decoder layer: one token each over the encoder's states
        dict(name="cross decode", op="attn", B=64, Hq=16, Hkv=16, D=64, ps=16, dtype="f16", P=0, plen=0, nlo=1, nhi=1,
             lo=1, hi=1500, causal=False),
        # the decoder's prompts over the encoder's states
        dict(name="cross prompts", op="attn", B=24, Hq=16, Hkv=16, D=64, ps=64, dtype="bf16", P=0, plen=0, nlo=3,
             nhi=448, lo=400, hi=1500, causal=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "append", "reserve", "attn", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "f16"])
    D = rng.choice([64, 128])
    ps = rng.choice([16, 32, 48, 64, 128, 208])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 6, 8, 12])
    if op == "reserve":
        B, hi, nhi = _log_int(rng, 1, 256), _log_int(rng, 1, 1500), _log_int(rng, 1, 600)
        pages = int(rng.uniform(1.05, 1.6) * B * (-(-(hi + nhi) // ps) + 1)) + rng.randrange(1, 50)
        return dict(op=op, B=B, ps=ps, n_pages=pages, nlo=rng.choice([0, 1, nhi]), nhi=nhi, lo=rng.choice([0, 1, hi]),
                    hi=hi)
    turn = dict(rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= D]), inter=rng.random() < 0.4,
                norm=rng.random() < 0.6, stretch=rng.choice([1.0, 1.0, 2.5, 8.0]), gate=rng.random() < 0.3)
    P = rng.choice([0, 0, 1, 1, 2])
    common = dict(op=op, Hq=G * Hkv, Hkv=Hkv, D=D, dtype=dtype, P=P)
    if op == "rope":
        K = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 12, 15, 16])
        B = _log_int(rng, 1, 256 // max(1, P)) * max(1, P)
        while B * K * (G + 2) * Hkv * D > 256 * 16 * 48 * 128:
            B = max(P, 1) * max(1, B // 2 // max(P, 1))
        hi = _log_int(rng, 1, 200000)
        return dict(common, B=B, K=K, plen=_log_int(rng, 1, 200000) if P else 0, lo=rng.choice([0, 1, hi]), hi=hi,
                    tree=rng.random() < 0.4, ragged=rng.random() < 0.4, **turn)
    B = _log_int(rng, 1, 64 // max(1, P)) * max(1, P)
    plen = _log_int(rng, 1, 2000) if P else 0
    if op == "append":
        hi, nhi = _log_int(rng, 1, 2000), _log_int(rng, 1, 8191)
        while B * nhi * (G + 2) * Hkv * D > 36000 * 48 * 128:
            nhi = (nhi + 1) // 2
        return dict(common, B=B, ps=ps, plen=plen, nlo=rng.choice([0, 1, nhi]), nhi=nhi, lo=rng.choice([0, 1, hi]),
                    hi=hi, **turn)
    causal = rng.random() < 0.7
    hi, nhi = _log_int(rng, 1, 60000 if B <= 2 else 3000), _log_int(rng, 1, 8000)
    # no more than the long prompts' products
    while B * nhi * (plen + hi + nhi) * G * Hkv * D > 1 << 40 or B * (hi + nhi) * Hkv * D > 1 << 28:
        plen, hi, nhi = (plen + 1) // 2, (hi + 1) // 2, (nhi + 1) // 2
    return dict(common, B=B, ps=ps, plen=plen, nlo=rng.choice([0, 1, nhi]), nhi=nhi, lo=rng.choice([0, 1, hi]), hi=hi,
                causal=causal)


# ------------------------------------------------------------------------------------- inputs
def _lens(lo, hi, n, rng):
    """n lengths spread evenly over lo..hi (their sum does not depend on the seed), in a random order."""
    return rng.permutation(np.linspace(lo, hi, n).round().astype(np.int64)) if n > 1 else np.array([hi])


def _gauss(shape, dtype, gen, scale=1.0):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.normal_(0.0, scale, generator=gen)
    return t


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _parents(B, K, rng):
    """Drafted trees: each node continues the node before it, or branches off an earlier one."""
    par = np.arange(K)[None, :].repeat(B, 0) - 1
    back = rng.integers(-1, np.maximum(1, np.arange(K))[None, :], (B, K))
    return np.where((rng.random((B, K)) < 0.4) & (np.arange(K)[None, :] > 0), np.minimum(back, par), par)


def _tables(pages, n_pages, width, rng):
    """Page tables of slots that own `pages` pages each, scattered over a pool as after long service."""
    ids = rng.permutation(n_pages)
    table = np.full((len(pages), width), -1, dtype=np.int64)
    table[np.arange(width)[None, :] < np.asarray(pages)[:, None]] = ids[:int(np.sum(pages))]
    return table


def _pages_of(lens, ps):
    return -(-np.asarray(lens) // ps)


def _frequencies(rot, stretch):
    """Radians a token of each pair; the slow pairs are slowed by `stretch`, the fast ones kept, with a ramp between."""
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    ramp = np.clip((np.arange(rot // 2) / (rot // 2) - 0.25) * 2.0, 0.0, 1.0)
    return f * (1.0 - ramp) + f / stretch * ramp


def _turning(c, gen):
    """What a layer keeps of its norms and its rotation."""
    w = [1.0 + 0.1 * torch.randn(c["D"], device="cuda", generator=gen) for _ in range(2)] if c["norm"] else [None, None]
    return dict(freq=torch.from_numpy(_frequencies(c["rot"], c["stretch"])).cuda(), q_weight=w[0], k_weight=w[1],
                eps=1e-6, magnitude=1.0 + 0.1 * math.log(c["stretch"]))


def _projection(c, n, dtype, gen):
    """q [n, Hq, D], k and v [n, Hkv, D]: parts of the rows of one projection (with `gate`, each query head's gate
    behind it)."""
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    wide = 2 if c["gate"] else 1
    x = _gauss((n, (Hq * wide + 2 * Hkv) * D), dtype, gen)
    q, k, v = x.split([Hq * wide * D, Hkv * D, Hkv * D], 1)
    return q.view(n, Hq, wide * D)[:, :, :D], k.view(n, Hkv, D), v.view(n, Hkv, D)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "dtype": _TYPES[case.get("dtype", "bf16")]}
    s.update({"rope": _prepare_rope, "append": _prepare_append, "reserve": _prepare_reserve,
              "attn": _prepare_attn}[case["op"]](case, s["dtype"], rng, gen))
    return s


def _prefix_of(c):
    return _i32(c["B"] + np.arange(c["B"]) // (c["B"] // c["P"])) if c["P"] else None


def _prepare_rope(c, dtype, rng, gen):
    B, K = c["B"], c["K"]
    lens = np.concatenate([_lens(c["lo"], c["hi"], B, rng), np.full(c["P"], c["plen"], dtype=np.int64)])
    q, k, v = (x.unflatten(0, (B, K)) for x in _projection(c, B * K, dtype, gen))
    return dict(q=q, k=k, v=v, lens=_i32(lens), prefix_of=_prefix_of(c),
                win_len=_i32(_lens(1, K, B, rng)) if c["ragged"] else None,
                parent=_i32(_parents(B, K, rng)) if c["tree"] else None,
                q_out=torch.empty((B, K, c["Hq"], c["D"]), dtype=dtype, device="cuda"),
                k_out=torch.empty((B, K, c["Hkv"], c["D"]), dtype=dtype, device="cuda"),
                v_out=torch.empty((B, K, c["Hkv"], c["D"]), dtype=dtype, device="cuda"), **_turning(c, gen))


def _ragged(c, rng, own_tokens):
    """Lengths of the slots with the new tokens, the packed tokens' bounds, page tables."""
    new, before = _lens(c["nlo"], c["nhi"], c["B"], rng), _lens(c["lo"], c["hi"], c["B"], rng)
    cu = np.concatenate([[0], np.cumsum(new)])
    lens = np.concatenate([before + new if own_tokens else before, np.full(c["P"], c["plen"], dtype=np.int64)])
    pages = _pages_of(lens, c["ps"])
    n_pages = int(lens.sum()) // c["ps"] + len(lens) + 8  # (enough for any order of the lengths)
    table = _tables(pages, n_pages, max(1, int(pages.max())), rng)
    return dict(cu=_i32(cu), bounds=cu.tolist(), n=int(cu[-1]), lens=_i32(lens), table=_i32(table),
                shape=(1, n_pages, c["ps"], c["Hkv"], c["D"]), prefix_of=_prefix_of(c))


def _prepare_append(c, dtype, rng, gen):
    s = _ragged(c, rng, True)
    q, k, v = _projection(c, s["n"], dtype, gen)
    s.update(q=q, k=k, v=v, k_cache=_gauss(s["shape"], dtype, gen), v_cache=_gauss(s["shape"], dtype, gen),
             q_out=torch.empty((s["n"], c["Hq"], c["D"]), dtype=dtype, device="cuda"), **_turning(c, gen))
    return s


def _prepare_attn(c, dtype, rng, gen):
    s = _ragged(c, rng, c["causal"])
    # trained attention is peaked: scores with a spread of a few units
    s.update(q=_gauss((s["n"], c["Hq"], c["D"]), dtype, gen, 2.0), k_cache=_gauss(s["shape"], dtype, gen),
             v_cache=_gauss(s["shape"], dtype, gen), scale=c["D"] ** -0.5, host_lens=s["lens"].tolist(),
             out=torch.empty((s["n"], c["Hq"], c["D"]), dtype=dtype, device="cuda"),
             lse=torch.empty((s["n"], c["Hq"]), dtype=torch.float32, device="cuda"))
    return s


def _prepare_reserve(c, dtype, rng, gen):
    new, before = _lens(c["nlo"], c["nhi"], c["B"], rng), _lens(c["lo"], c["hi"], c["B"], rng)
    pages = _pages_of(before, c["ps"])
    table = _tables(pages, c["n_pages"], -(-(c["hi"] + c["nhi"]) // c["ps"]) + 1, rng)
    ref = np.bincount(table[table >= 0].ravel(), minlength=c["n_pages"])
    s = dict(new=_i32(new), table=_i32(table), lens=_i32(before), ref=_i32(ref))
    s.update(table_out=torch.empty_like(s["table"]), lens_out=torch.empty_like(s["lens"]),
             ref_out=torch.empty_like(s["ref"]))
    return s


# ------------------------------------------------------------------------------------- passes
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "reserve": _own_reserve, "attn": _own_attn}[op](s)
    return {"rope": _plain_rope, "append": _plain_append, "reserve": _plain_reserve, "attn": _plain_attn}[op](s)


def _handle(s):
    """Shapes, norms and rotation, and workspace of the library's calls: kept by a user's program beside its cache."""
    if "handle" not in s:
        from speculative_decode_verify_gdn_gb300 import kv
        c = s["case"]
        op = c["op"]
        rope = kv.make_rope(c["D"], s["freq"], interleaved=c["inter"], magnitude=s["magnitude"], q_weight=s["q_weight"],
                            k_weight=s["k_weight"], eps=s["eps"]) if op in ("rope", "append") else None
        pool = s.get("k_cache")
        dims = kv.make_kv_dims(B=c["B"], K=c.get("K", 1), Hq=c.get("Hq", 1), Hkv=c.get("Hkv", 1), D=c.get("D", 64),
                               page_size=c.get("ps", 16), n_pages=pool.shape[1] if pool is not None else c.get("n_pages", 1),
                               max_pages=s["table"].shape[1] if "table" in s else 1 << 16, n_slots=s["lens"].shape[0],
                               dtype=s["dtype"])
        ws = kv.alloc_kv_workspace(dims) if op == "reserve" else \
            kv.alloc_attn_prefill_workspace(dims, s["n"]) if op == "attn" else None
        s["handle"] = kv, dims, rope, ws
    return s["handle"]


def _own_rope(s):
    kv, dims, rope, _ = _handle(s)
    kv.gdn_attn_rope(dims, rope, s["q"], s["k"], s["v"], s["lens"], s["prefix_of"], s["win_len"], s["parent"], None,
                     s["q_out"], s["k_out"], s["v_out"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_append(s):
    kv, dims, rope, _ = _handle(s)
    kv.gdn_kv_append(dims, 0, rope, s["cu"], s["q"], s["k"], s["v"], None, s["k_cache"], s["v_cache"], s["table"],
                     s["lens"], s["prefix_of"], s["q_out"])
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _own_reserve(s):
    kv, dims, _, ws = _handle(s)
    kv.gdn_kv_reserve(dims, s["new"], s["table"], s["table_out"], s["lens"], s["lens_out"], s["ref"], s["ref_out"], ws)
    return {"table": s["table_out"], "lens": s["lens_out"], "ref": s["ref_out"]}


def _own_attn(s):
    kv, dims, _, ws = _handle(s)
    kv.gdn_attn_prefill(dims, 0, s["cu"], s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["prefix_of"],
                        s["case"]["causal"], s["scale"], s["out"], s["lse"], ws)
    return {"out": s["out"], "lse": s["lse"]}


def _turned(x, weight, cos, sin, s):
    """x [..., H, D] in 32 bits, normed and rotated; cos, sin [..., 1, rot / 2]."""
    rot, x = s["case"]["rot"], x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["case"]["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1 if s["case"]["inter"] else -2).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1).to(s["dtype"])


def _angles(pos, s):
    """Far positions take their angles in 64 bits."""
    angle = (pos.double()[..., None] * s["freq"])[..., None, :]
    return (torch.cos(angle) * s["magnitude"]).float(), (torch.sin(angle) * s["magnitude"]).float()


def _before(s):
    """Tokens of each sequence's prefix."""
    return 0 if s["prefix_of"] is None else s["lens"][s["prefix_of"].long()].long()


def _depths(parent, B, K, device):
    """Tokens above each node (powers of the parent matrix, which is nilpotent)."""
    node = torch.arange(K, device=device)
    if parent is None:
        return node.expand(B, K)
    p = (parent[:, :, None] == node).float()
    eye, p2 = torch.eye(K, device=device), p @ p
    p4 = p2 @ p2
    return (((eye + p) @ (eye + p2) @ (eye + p4) @ (eye + p4 @ p4)) > 0.5).sum(-1) - 1


def _plain_rope(s):
    c = s["case"]
    B, K, dev = c["B"], c["K"], s["lens"].device
    pos = (s["lens"][:B].long() + _before(s))[:, None] + _depths(s["parent"], B, K, dev)
    cos, sin = _angles(pos, s)
    q, k, v = _turned(s["q"], s["q_weight"], cos, sin, s), _turned(s["k"], s["k_weight"], cos, sin, s), s["v"]
    if s["win_len"] is not None:  # padding tokens are 0
        live = (torch.arange(K, device=dev) < s["win_len"][:, None])[:, :, None, None]
        q, k, v = (torch.where(live, x, 0.0) for x in (q, k, v))
    return {"q": q, "k": k, "v": v}


def _plain_append(s):
    c = s["case"]
    B, dev = c["B"], s["lens"].device
    cu, lens = s["cu"].long(), s["lens"][:B].long()
    at = torch.arange(s["n"], device=dev)
    seq = torch.searchsorted(cu, at, right=True) - 1
    own_pos = lens[seq] - cu[seq + 1] + at
    pos = own_pos if s["prefix_of"] is None else own_pos + _before(s)[seq]
    cos, sin = _angles(pos, s)
    page, row = s["table"][seq, own_pos // c["ps"]].long(), own_pos % c["ps"]
    s["k_cache"][0, page, row] = _turned(s["k"], s["k_weight"], cos, sin, s)
    s["v_cache"][0, page, row] = s["v"]
    return {"q": _turned(s["q"], s["q_weight"], cos, sin, s), "k": s["k_cache"], "v": s["v_cache"]}


def _plain_reserve(s):
    ps, ref = s["case"]["ps"], s["ref"]
    lens = s["lens"].long()
    grown = lens + s["new"].long()
    have, want = (lens + ps - 1) // ps, (grown + ps - 1) // ps
    need = want - have
    first = torch.cumsum(need, 0) - need
    ids = torch.nonzero(ref == 0)[:, 0]  # the lowest free pages go to the lowest sequences
    col = torch.arange(s["table"].shape[1], device=ref.device)
    fresh = (col >= have[:, None]) & (col < want[:, None])
    table = torch.where(fresh, ids[(first[:, None] + col - have[:, None]).clamp(0, ids.numel() - 1)], s["table"].long())
    out = ref.clone()
    out[table[fresh]] = 1
    return {"table": table.int(), "lens": grown.int(), "ref": out}


def _tokens(cache, table, slot, n, ps):
    return cache[0].index_select(0, table[slot, :-(-n // ps)]).flatten(0, 1)[:n]


def _plain_attn(s):
    """A sequence, a stretch of its rows and a few key/value heads at a time, with the scores of all their keys."""
    c = s["case"]
    B, Hq, Hkv, D, ps, lens, bounds = c["B"], c["Hq"], c["Hkv"], c["D"], c["ps"], s["host_lens"], s["bounds"]
    G, out, lse = Hq // Hkv, torch.zeros_like(s["out"]), torch.full_like(s["lse"], -math.inf)
    for b in range(B):
        n, m = bounds[b + 1] - bounds[b], lens[b]
        pre = lens[B + b // (B // c["P"])] if c["P"] else 0
        if n == 0 or pre + m == 0:
            continue
        k, v = (torch.cat(([_tokens(x, s["table"], B + b // (B // c["P"]), pre, ps)] if pre else []) +
                          ([_tokens(x, s["table"], b, m, ps)] if m else [])).float().transpose(0, 1)
                for x in (s["k_cache"], s["v_cache"]))
        rows = max(1, min(n, 2048))
        for r0 in range(0, n, rows):
            r1 = min(n, r0 + rows)
            seen = pre + m - n + r1 if c["causal"] else pre + m  # the last row's keys
            q = s["q"][bounds[b] + r0:bounds[b] + r1].float() * s["scale"]
            q = q.view(r1 - r0, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * (r1 - r0), D)
            step = max(1, min(Hkv, (1 << 29) // (G * (r1 - r0) * seen)))
            for h in range(0, Hkv, step):
                x = q[h:h + step] @ k[h:h + step, :seen].transpose(1, 2)
                if c["causal"]:
                    limit = torch.arange(seen - (r1 - r0), seen, device=x.device).repeat(G)[:, None]
                    x = torch.where(torch.arange(seen, device=x.device) <= limit, x, -math.inf)
                top = x.amax(-1, keepdim=True)
                x = torch.exp(x - top)
                total = x.sum(-1, keepdim=True)
                hs = x.shape[0]
                o = ((x @ v[h:h + step, :seen]) / total).view(hs, G, r1 - r0, D).permute(2, 0, 1, 3)
                at, heads = slice(bounds[b] + r0, bounds[b] + r1), slice(h * G, (h + hs) * G)
                out[at, heads] = o.flatten(1, 2).to(s["dtype"])
                lse[at, heads] = (top + torch.log(total)).view(hs, G, r1 - r0).permute(2, 0, 1).flatten(1, 2)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """Straight from the definitions, in float64 (reserve counts pages, and computes no numbers)."""
    if case["op"] == "reserve" or (case["op"] == "attn" and work(case)["flops"] > 1e13):
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn}[case["op"]](case, s)


def _turn64(x, weight, position, c, s):
    """x [H, D] at one position, or [n, H, D] at n of them: complex numbers times unit ones."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + s["eps"]).sqrt() * weight.double()
    head, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    z = head.unflatten(-1, (-1, 2)) if c["inter"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.complex(z[..., 0], z[..., 1])
    angle = torch.as_tensor(position, dtype=torch.float64, device=x.device)[..., None, None] * s["freq"]
    z = torch.view_as_real(z * torch.polar(torch.full_like(angle, s["magnitude"]), angle))
    return torch.cat([(z if c["inter"] else z.transpose(-1, -2)).flatten(-2), rest], -1)


def _exact_rope(c, s):
    B, K = c["B"], c["K"]
    lens = s["lens"].tolist()
    prefix = s["prefix_of"].tolist() if c["P"] else None
    parent = s["parent"].tolist() if c["tree"] else None
    win = s["win_len"].tolist() if c["ragged"] else [K] * B
    position, live = torch.zeros((B, K), dtype=torch.float64), torch.zeros((B, K, 1, 1), dtype=torch.float64)
    for b in range(B):
        depth = []
        for t in range(K):
            up = t - 1 if parent is None else parent[b][t]
            depth.append(0 if up < 0 else depth[up] + 1)
            position[b, t] = lens[b] + depth[t] + (lens[prefix[b]] if prefix else 0)
            live[b, t] = float(t < win[b])
    live = live.cuda()
    return {"q": _turn64(s["q"], s["q_weight"], position.cuda(), c, s) * live,
            "k": _turn64(s["k"], s["k_weight"], position.cuda(), c, s) * live, "v": s["v"].double() * live}


def _exact_append(c, s):
    lens, prefix, table = s["lens"].tolist(), s["prefix_of"].tolist() if c["P"] else None, s["table"].long()
    q, k, v = torch.zeros_like(s["q_out"], dtype=torch.float64), s["k_cache"].double(), s["v_cache"].double()
    for b in range(c["B"]):
        lo, hi = s["bounds"][b], s["bounds"][b + 1]
        own = torch.arange(lens[b] - (hi - lo), lens[b], device="cuda")
        position = own + (lens[prefix[b]] if prefix else 0)
        q[lo:hi] = _turn64(s["q"][lo:hi], s["q_weight"], position, c, s)
        page, row = table[b].index_select(0, own // c["ps"]), own % c["ps"]
        k[0, page, row] = _turn64(s["k"][lo:hi], s["k_weight"], position, c, s)
        v[0, page, row] = s["v"][lo:hi].double()
    return {"q": q, "k": k, "v": v}


def _exact_attn(c, s):
    lens, table, ps = s["lens"].tolist(), s["table"].tolist(), c["ps"]
    prefix = s["prefix_of"].tolist() if c["P"] else None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")

    def rows(cache, slot):
        ids = torch.tensor(table[slot][:-(-lens[slot] // ps)], dtype=torch.long, device="cuda")
        return cache[0][ids].flatten(0, 1)[:lens[slot]]

    for b in range(c["B"]):
        lo, hi = s["bounds"][b], s["bounds"][b + 1]
        slots = ([prefix[b]] if prefix else []) + [b]
        k, v = (torch.cat([rows(x, i) for i in slots]) for x in (s["k_cache"], s["v_cache"]))
        if hi == lo or k.shape[0] == 0:
            continue
        for h in range(c["Hq"]):
            kh, vh = (x[:, h * c["Hkv"] // c["Hq"]].double() for x in (k, v))
            for r in range(lo, hi, 4096):
                e = min(hi, r + 4096)
                n = kh.shape[0] - (hi - e) if c["causal"] else kh.shape[0]
                x = s["q"][r:e, h].double() @ kh[:n].T * s["scale"]
                if c["causal"]:
                    x = x.masked_fill(torch.ones_like(x, dtype=torch.bool).triu(n - (e - r) + 1), -math.inf)
                lse[r:e, h] = torch.logsumexp(x, -1)
                out[r:e, h] = torch.softmax(x, -1) @ vh[:n]
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------- work
def work(case):
    c = case
    rng = np.random.default_rng(0)
    if c["op"] == "reserve":
        width = -(-(c["hi"] + c["nhi"]) // c["ps"]) + 1
        return {"bytes": 8 * (c["n_pages"] + c["B"] * (width + 1)), "flops": 0}
    row = 2 * c["D"]
    if c["op"] == "rope":
        n = int(_lens(1, c["K"], c["B"], rng).sum()) if c["ragged"] else c["B"] * c["K"]
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": row * heads * (n + c["B"] * c["K"]), "flops": 6.0 * c["D"] * heads * n}
    new = int(_lens(c["nlo"], c["nhi"], c["B"], rng).sum())
    if c["op"] == "append":
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": 2 * row * heads * new, "flops": 6.0 * c["D"] * heads * new}
    old = int(_lens(c["lo"], c["hi"], c["B"], rng).sum())
    n = _lens(c["nlo"], c["nhi"], c["B"], rng).astype(float)
    if c["causal"]:
        seen = float((n * (c["plen"] * (c["P"] > 0) + old / c["B"] + (n + 1) / 2)).sum())
    else:
        seen = float((n * (c["plen"] * (c["P"] > 0) + old / c["B"])).sum())
    states = c["P"] * c["plen"] + old + (new if c["causal"] else 0)
    return {"bytes": 2 * row * c["Hkv"] * states + new * c["Hq"] * (2 * row + 4), "flops": 4.0 * c["D"] * c["Hq"] * seen}
