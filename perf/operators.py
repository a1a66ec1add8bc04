"""Cases of the paged key/value cache operators: attention of a verify window over a cache whose
sequences share long prefixes, and the cache's own upkeep (commit, fork, compact).

These are the softmax-attention layers' half of a speculative-decoding round in a hybrid model
whose linear-attention half is the gated delta rule: the window's K drafted tokens attend to the
shared prefix, to their own sequence and to each other; the accepted ones are then committed to
pages; sequences are forked and dropped; and the pool is compacted.

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
        # one user, plain decode of a hybrid model's attention layer: the latency end
        dict(name="attn one decode token", op="attn", B=1, K=1, Hq=16, Hkv=2, D=128, ps=16, dtype="bf16",
             P=0, plen=0, lo=700, hi=700, tree=False, ragged=False),
        # a small ragged batch of drafted token trees behind one system prompt, padded windows, f16
        dict(name="attn ragged trees", op="attn", B=13, K=7, Hq=24, Hkv=4, D=64, ps=48, dtype="f16",
             P=1, plen=1531, lo=0, hi=901, tree=True, ragged=True),
        # the serving verify batch (B=32, K=16) behind a long system prompt
        dict(name="attn serving verify", op="attn", B=32, K=16, Hq=32, Hkv=8, D=128, ps=64, dtype="bf16",
             P=1, plen=8192, lo=1, hi=2048, tree=False, ragged=False),
        # one long conversation, a window of 16 drafted tokens: few rows, a long axis to split
        dict(name="attn one long sequence", op="attn", B=1, K=16, Hq=32, Hkv=8, D=128, ps=64, dtype="bf16",
             P=0, plen=0, lo=131072, hi=131072, tree=False, ragged=False),
        # plain decode of many users of four applications, each with its own prompt
        dict(name="attn many decodes", op="attn", B=256, K=1, Hq=32, Hkv=8, D=128, ps=16, dtype="bf16",
             P=4, plen=3001, lo=5, hi=1024, tree=False, ragged=False),
        # a wide verify batch over one document of 32k tokens: the matrix-product end
        dict(name="attn document batch", op="attn", B=64, K=16, Hq=32, Hkv=4, D=128, ps=64, dtype="bf16",
             P=1, plen=32768, lo=1, hi=512, tree=True, ragged=False),
        # one user's accepted draft, a few layers
        dict(name="commit one sequence", op="commit", B=1, K=4, Hkv=2, D=128, ps=16, dtype="bf16", layers=4,
             n_pages=256, lo=700, hi=700, tree=False),
        # the serving batch's accepted tree paths in all 12 attention layers of a 48-layer hybrid stack
        dict(name="commit serving batch", op="commit", B=256, K=16, Hkv=8, D=128, ps=16, dtype="bf16", layers=12,
             n_pages=5000, lo=1, hi=400, tree=True),
        # one sequence resampled into four
        dict(name="fork one into four", op="fork", slots=4, Hkv=2, D=64, ps=16, dtype="f16", layers=4,
             n_pages=200, lo=37, hi=300),
        # a population of sequences resampled: some dropped, some taken many times
        dict(name="fork a population", op="fork", slots=192, Hkv=8, D=128, ps=64, dtype="bf16", layers=12,
             n_pages=1500, lo=1, hi=400),
        # a small pool made dense
        dict(name="compact a small pool", op="compact", slots=7, Hkv=2, D=64, ps=16, dtype="bf16", layers=4,
             n_pages=333, live=0.5),
        # a full-sized pool made dense after many sequences ended
        dict(name="compact a large pool", op="compact", slots=128, Hkv=8, D=128, ps=16, dtype="bf16", layers=12,
             n_pages=4500, live=0.6),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "commit", "fork", "compact"])
    dtype = rng.choice(["bf16", "f16"])
    D = rng.choice([64, 128])
    ps = rng.choice([16, 32, 48, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "attn":
        G = rng.choice([1, 2, 3, 4, 6, 8])
        K = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 12, 15, 16])
        P = rng.choice([0, 1, 1, 1, 2, 3])
        per = _log_int(rng, 1, 96 // max(1, P))
        B = per * max(1, P)
        hi = _log_int(rng, 1, 4096 if B > 4 else 100000)
        plen = _log_int(rng, 1, 32768) if P else 0
        # no more than the document batch: its rows times its keys, and a plain pass that fits
        while B * K * G * Hkv * max(1, plen + hi) > 64 * 16 * 32 * 32768 or B * hi * Hkv * D > 1 << 29:
            plen, hi = (plen + 1) // 2, (hi + 1) // 2
        return dict(op="attn", B=B, K=K, Hq=G * Hkv, Hkv=Hkv, D=D, ps=ps, dtype=dtype, P=P, plen=plen,
                    lo=rng.choice([0, 1, hi]), hi=hi, tree=rng.random() < 0.4, ragged=rng.random() < 0.4)
    layers = rng.choice([1, 2, 4, 12])
    if op == "commit":
        B, K, hi = _log_int(rng, 1, 256), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 15, 16]), _log_int(rng, 1, 600)
        pages = int(1.3 * B * (-(-(hi + K) // ps) + 1)) + rng.randrange(1, 50)
        while layers * pages * ps * Hkv * D > 900_000_000:
            layers = max(1, layers // 2)
            if layers == 1:
                Hkv = max(1, Hkv // 2)
            if layers == 1 and Hkv == 1:
                break
        return dict(op="commit", B=B, K=K, Hkv=Hkv, D=D, ps=ps, dtype=dtype, layers=layers, n_pages=pages,
                    lo=rng.choice([0, 1, hi]), hi=hi, tree=rng.random() < 0.5)
    if op == "fork":
        slots, hi = _log_int(rng, 2, 192), _log_int(rng, 1, 600)
        pages = int(1.2 * slots * (-(-hi // ps) + 1)) + rng.randrange(1, 50)
        while layers * pages * ps * Hkv * D > 900_000_000:
            layers = max(1, layers // 2)
            if layers == 1:
                Hkv = max(1, Hkv // 2)
        return dict(op="fork", slots=slots, Hkv=Hkv, D=D, ps=ps, dtype=dtype, layers=layers, n_pages=pages,
                    lo=rng.choice([0, 1, hi]), hi=hi)
    pages = _log_int(rng, 40, 8000)
    while layers * pages * ps * Hkv * D > 850_000_000:
        pages = (2 * pages) // 3
    return dict(op="compact", slots=_log_int(rng, 1, 128), Hkv=Hkv, D=D, ps=ps, dtype=dtype, layers=layers,
                n_pages=pages, live=rng.uniform(0.1, 0.95))


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


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "dtype": _TYPES[case["dtype"]]}
    s.update({"attn": _prepare_attn, "commit": _prepare_commit, "fork": _prepare_fork,
              "compact": _prepare_compact}[case["op"]](case, s["dtype"], rng, gen))
    return s


def _pages_of(lens, ps):
    return -(-np.asarray(lens) // ps)


def _tables(pages, n_pages, width, rng):
    """Page tables of slots that own `pages` pages each, scattered over a pool as after long service."""
    ids = rng.permutation(n_pages)
    table = np.full((len(pages), width), -1, dtype=np.int64)
    table[np.arange(width)[None, :] < np.asarray(pages)[:, None]] = ids[:int(np.sum(pages))]
    return table


def _prepare_attn(c, dtype, rng, gen):
    B, K, P = c["B"], c["K"], c["P"]
    lens = np.concatenate([_lens(c["lo"], c["hi"], B, rng), np.full(P, c["plen"], dtype=np.int64)])
    pages = _pages_of(lens, c["ps"])
    n_pages = int(pages.sum()) + 8
    width = max(1, int(pages.max()))
    shape = (1, n_pages, c["ps"], c["Hkv"], c["D"])
    win = _lens(1, K, B, rng) if c["ragged"] else np.full(B, K)
    return dict(
        # trained attention is peaked: scores with a spread of a few units
        q=_gauss((B, K, c["Hq"], c["D"]), dtype, gen, 2.0),
        k_win=_gauss((B, K, c["Hkv"], c["D"]), dtype, gen), v_win=_gauss((B, K, c["Hkv"], c["D"]), dtype, gen),
        k_cache=_gauss(shape, dtype, gen), v_cache=_gauss(shape, dtype, gen),
        table=_i32(_tables(pages, n_pages, width, rng)), lens=_i32(lens),
        prefix_of=_i32(B + np.arange(B) // (B // P)) if P else None,
        win_len=_i32(win) if c["ragged"] else None,
        parent=_i32(_parents(B, K, rng)) if c["tree"] else None, scale=c["D"] ** -0.5,
        out=torch.empty((B, K, c["Hq"], c["D"]), dtype=dtype, device="cuda"),
        lse=torch.empty((B, K, c["Hq"]), dtype=torch.float32, device="cuda"))


def _pool(c, dtype, gen):
    shape = (c["layers"], c["n_pages"], c["ps"], c["Hkv"], c["D"])
    return dict(k_cache=_gauss(shape, dtype, gen), v_cache=_gauss(shape, dtype, gen))


def _bookkeeping(table, lens, n_pages):
    ref = np.bincount(table[table >= 0].ravel(), minlength=n_pages)
    t = dict(table=_i32(table), lens=_i32(lens), ref=_i32(ref))
    t.update(table_out=torch.empty_like(t["table"]), lens_out=torch.empty_like(t["lens"]),
             ref_out=torch.empty_like(t["ref"]))
    return t


def _prepare_commit(c, dtype, rng, gen):
    B, K = c["B"], c["K"]
    lens = _lens(c["lo"], c["hi"], B, rng)
    pages = _pages_of(lens, c["ps"])
    width = int(_pages_of(lens + K, c["ps"]).max())
    s = _pool(c, dtype, gen)
    s.update(_bookkeeping(_tables(pages, c["n_pages"], width, rng), lens, c["n_pages"]))
    win = (c["layers"], B, K, c["Hkv"], c["D"])
    s.update(k_win=_gauss(win, dtype, gen), v_win=_gauss(win, dtype, gen), accept=_i32(_lens(1, K, B, rng)),
             parent=_i32(_parents(B, K, rng)) if c["tree"] else None)
    return s


def _prepare_fork(c, dtype, rng, gen):
    n = c["slots"]
    lens = _lens(c["lo"], c["hi"], n, rng)
    pages = _pages_of(lens, c["ps"])
    # resampling by weight: heavy sequences are taken again and again, light ones die out
    src = np.sort(rng.choice(n, n, p=rng.dirichlet(np.full(n, 0.7))))
    src[rng.random(n) < 0.05] = -1
    s = _pool(c, dtype, gen)
    s.update(_bookkeeping(_tables(pages, c["n_pages"], int(pages.max()) + 1, rng), lens, c["n_pages"]))
    s["src"] = _i32(src)
    return s


def _prepare_compact(c, dtype, rng, gen):
    n = c["slots"]
    live = max(1, int(c["live"] * c["n_pages"]))
    pages = np.linspace(0, 2 * live / n, n).astype(np.int64)  # short and long sequences alike
    pages[-1] += live - pages.sum()
    pages = rng.permutation(pages)
    lens = np.maximum(0, pages * c["ps"] - rng.integers(0, c["ps"], n))
    table = _tables(pages, c["n_pages"], int(pages.max()), rng)
    s = _pool(c, dtype, gen)
    s.update(_bookkeeping(table, lens, c["n_pages"]))
    s["n_live"] = torch.empty(1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------- passes
def run(s):
    op = s["case"]["op"]
    if own:
        return {"attn": _own_attn, "commit": _own_commit, "fork": _own_fork, "compact": _own_compact}[op](s)
    return {"attn": _plain_attn, "commit": _plain_commit, "fork": _plain_fork, "compact": _plain_compact}[op](s)


def _handle(s):
    """Shapes and workspace of the library's calls, kept by a user's program beside its cache."""
    if "handle" not in s:
        from speculative_decode_verify_gdn_gb300 import kv
        c = s["case"]
        attn = c["op"] == "attn"
        dims = kv.make_kv_dims(B=c.get("B", 0), K=c.get("K", 1), Hq=c.get("Hq", c["Hkv"]), Hkv=c["Hkv"], D=c["D"],
                               page_size=c["ps"], n_pages=s["k_cache"].shape[1], max_pages=s["table"].shape[1],
                               n_slots=s["table"].shape[0], n_layers=s["k_cache"].shape[0], dtype=s["dtype"])
        s["handle"] = kv, dims, (kv.alloc_attn_workspace if attn else kv.alloc_kv_workspace)(dims)
    return s["handle"]


def _own_attn(s):
    kv, dims, ws = _handle(s)
    kv.gdn_attn_verify(dims, 0, s["q"], s["k_win"], s["v_win"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                       s["prefix_of"], s["win_len"], s["parent"], s["scale"], s["out"], s["lse"], ws)
    return {"out": s["out"], "lse": s["lse"]}


def _own_commit(s):
    kv, dims, ws = _handle(s)
    kv.gdn_kv_commit(dims, s["accept"], s["parent"], s["k_win"], s["v_win"], s["k_cache"], s["v_cache"], s["table"],
                     s["table_out"], s["lens"], s["lens_out"], s["ref"], s["ref_out"], ws)
    return {"k": s["k_cache"], "v": s["v_cache"], "table": s["table_out"], "lens": s["lens_out"], "ref": s["ref_out"]}


def _own_fork(s):
    kv, dims, ws = _handle(s)
    kv.gdn_kv_fork(dims, s["src"], s["k_cache"], s["v_cache"], s["table"], s["table_out"], s["lens"], s["lens_out"],
                   s["ref"], s["ref_out"], ws)
    return {"k": s["k_cache"], "v": s["v_cache"], "table": s["table_out"], "lens": s["lens_out"], "ref": s["ref_out"]}


def _own_compact(s):
    kv, dims, ws = _handle(s)
    kv.gdn_kv_compact(dims, s["k_cache"], s["v_cache"], s["table"], s["table_out"], s["lens"], s["ref"], s["ref_out"],
                      s["n_live"], ws)
    return {"k": s["k_cache"], "v": s["v_cache"], "table": s["table_out"], "ref": s["ref_out"], "n_live": s["n_live"]}


def _ancestors(parent, B, K, device):
    """[B, K, K] bool: node j is node t or above it ((I - P)^-1 of the parent matrix P, nilpotent)."""
    if parent is None:
        return torch.ones((K, K), dtype=torch.bool, device=device).tril()[None].expand(B, K, K)
    node = torch.arange(K, device=device)
    p = (parent[:, :, None] == node).float()
    eye = torch.eye(K, device=device)
    p2 = p @ p
    p4 = p2 @ p2
    return ((eye + p) @ (eye + p2) @ (eye + p4) @ (eye + p4 @ p4)) > 0.5


def _plain_attn(s):
    c = s["case"]
    B, K, Hq, Hkv, D, P, ps = c["B"], c["K"], c["Hq"], c["Hkv"], c["D"], c["P"], c["ps"]
    G, dev = Hq // Hkv, s["q"].device
    q = s["q"].float().view(B, K, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, K * G, D) * s["scale"]
    lens = s["lens"].long()
    node = torch.arange(K, device=dev)
    low = float("-inf")

    def cached(rows, n):
        cols = max(1, -(-n // ps))
        at = s["table"][rows, :cols].long().clamp(min=0)
        k, v = (t[0][at].float().reshape(at.shape[0], cols * ps, Hkv, D).transpose(1, 2)
                for t in (s["k_cache"], s["v_cache"]))
        return k, v, (torch.arange(cols * ps, device=dev) < lens[rows][:, None])[:, None, None, :]

    k, v, seen = cached(slice(0, B), c["hi"])
    scores = [torch.where(seen, q @ k.transpose(-1, -2), low)]
    values = [v]
    kw, vw = (s[x].float().transpose(1, 2) for x in ("k_win", "v_win"))
    win_len = s["win_len"].long() if s["win_len"] is not None else torch.full((B,), K, device=dev)
    seen = _ancestors(s["parent"], B, K, dev) & (node < win_len[:, None])[:, None, :]
    seen = seen[:, None, :, None, :].expand(B, 1, K, G, K).reshape(B, 1, K * G, K)
    scores.append(torch.where(seen, q @ kw.transpose(-1, -2), low))
    values.append(vw)
    if P:
        per = B // P
        k, v, seen = cached(slice(B, B + P), c["plen"])
        qp = q.view(P, per, Hkv, K * G, D).transpose(1, 2).reshape(P, Hkv, per * K * G, D)
        sp = torch.where(seen, qp @ k.transpose(-1, -2), low)
        scores.append(sp.view(P, Hkv, per, K * G, -1).transpose(1, 2).reshape(B, Hkv, K * G, -1))
        values.append(v)
    m = torch.stack([x.amax(-1, keepdim=True) for x in scores]).amax(0)
    probs = [torch.exp(x - m) for x in scores]
    total = torch.stack([x.sum(-1, keepdim=True) for x in probs]).sum(0)
    acc = probs[0] @ values[0] + probs[1] @ values[1]
    if P:
        pp = probs[2].view(P, per, Hkv, K * G, -1).transpose(1, 2).reshape(P, Hkv, per * K * G, -1)
        acc = acc + (pp @ values[2]).view(P, Hkv, per, K * G, D).transpose(1, 2).reshape(B, Hkv, K * G, D)
    live = (node < win_len[:, None])[:, :, None, None]  # a padding token's row is 0 and -inf
    o = (acc / total).view(B, Hkv, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, Hq, D)
    lse = (m + torch.log(total)).view(B, Hkv, K, G).permute(0, 2, 1, 3).reshape(B, K, Hq)
    return {"out": torch.where(live, o, 0.0).to(s["dtype"]), "lse": torch.where(live[..., 0], lse, low)}


def _free_ids(ref, n):
    """The n lowest page ids that nothing refers to (n_pages where there are fewer)."""
    free = ref == 0
    rank = torch.cumsum(free, 0) - 1
    ids = torch.full((n + 1,), ref.numel(), dtype=torch.long, device=ref.device)
    ids.scatter_(0, torch.where(free & (rank < n), rank, n), torch.arange(ref.numel(), device=ref.device))
    return ids[:n]


def _plain_commit(s):
    c = s["case"]
    B, K, ps = c["B"], c["K"], c["ps"]
    dev, lens = s["lens"].device, s["lens"].long()
    anc = _ancestors(s["parent"], B, K, dev)
    accept = s["accept"].long()
    node = torch.arange(K, device=dev)
    path = anc[torch.arange(B, device=dev), (accept - 1).clamp(min=0)] & (accept > 0)[:, None]
    new = lens + path.sum(1)
    have, want = (lens + ps - 1) // ps, (new + ps - 1) // ps
    need = want - have
    first = torch.cumsum(need, 0) - need
    width = s["table"].shape[1]
    col = torch.arange(width, device=dev)
    fresh = (col >= have[:, None]) & (col < want[:, None])
    ids = _free_ids(s["ref"], B * (-(-K // ps) + 1))
    table = torch.where(fresh, ids[(first[:, None] + col - have[:, None]).clamp(0, ids.numel() - 1)], s["table"].long())
    ref = s["ref"].clone()
    ref[table[fresh]] = 1
    b, t = torch.nonzero(path, as_tuple=True)
    at = lens[b] + (torch.cumsum(path, 1) - 1)[b, t]
    page, row = table[b, at // ps], at % ps
    s["k_cache"][:, page, row] = s["k_win"][:, b, t]
    s["v_cache"][:, page, row] = s["v_win"][:, b, t]
    return {"k": s["k_cache"], "v": s["v_cache"], "table": table.int(), "lens": new.int(), "ref": ref}


def _plain_fork(s):
    c = s["case"]
    n, ps = c["slots"], c["ps"]
    dev, lens, src = s["lens"].device, s["lens"].long(), s["src"].long()
    slot = torch.arange(n, device=dev)
    used = src >= 0
    at = src.clamp(min=0)
    first = torch.full((n + 1,), n, device=dev).scatter_reduce_(0, torch.where(used, src, n), slot, "amin")[:n]
    new = torch.where(used, lens[at], 0)
    copy = used & (first[at] != slot) & (new % ps != 0)
    ids = _free_ids(s["ref"], n)[(torch.cumsum(copy, 0) - 1).clamp(min=0)]
    last = (new // ps).clamp(max=s["table"].shape[1] - 1)
    col = torch.arange(s["table"].shape[1], device=dev)
    table = torch.where(used[:, None], s["table"].long()[at], -1)
    old = table[slot, last]
    table = torch.where(copy[:, None] & (col == last[:, None]), ids[:, None], table)

    def count(tab, ln):
        held = (col < ((ln + ps - 1) // ps)[:, None]).int()
        return torch.zeros(c["n_pages"], dtype=torch.int32, device=dev).scatter_add_(
            0, tab.clamp(min=0).reshape(-1), held.reshape(-1))

    ref = s["ref"] - count(s["table"].long(), lens) + count(table, new)
    i = torch.nonzero(copy)[:, 0]
    row = torch.arange(ps, device=dev)
    keep = (row < (new[i] % ps)[:, None])[None, :, :, None, None]
    for x in (s["k_cache"], s["v_cache"]):
        x[:, table[i, last[i]]] = torch.where(keep, x[:, old[i]], x[:, table[i, last[i]]])
    return {"k": s["k_cache"], "v": s["v_cache"], "table": table.int(), "lens": new.int(), "ref": ref}


def _plain_compact(s):
    ref = s["ref"]
    n = ref.numel()
    live = ref > 0
    total = live.sum()
    page = torch.arange(n, device=ref.device)
    moves, holes = live & (page >= total), ~live & (page < total)
    source, target = torch.nonzero(moves)[:, 0], torch.nonzero(holes)[:, 0]
    where = page.clone()
    where[source] = target
    held = torch.arange(s["table"].shape[1], device=ref.device) < (
        (s["lens"] + s["case"]["ps"] - 1) // s["case"]["ps"])[:, None]
    table = torch.where(held, where[s["table"].long().clamp(min=0)], s["table"].long())
    ref_out = torch.where(moves, 0, ref)
    ref_out[target] = ref[source]
    s["k_cache"][:, target] = s["k_cache"][:, source]
    s["v_cache"][:, target] = s["v_cache"][:, source]
    return {"k": s["k_cache"], "v": s["v_cache"], "table": table.int(), "ref": ref_out, "n_live": total.int()[None]}


# ------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """Attention straight from its definition, one sequence at a time, in float64; the cache's
    upkeep moves values and counts, and computes none."""
    if case["op"] != "attn":
        return None
    s = prepare(case, seed)
    B, K, Hq, Hkv, ps = case["B"], case["K"], case["Hq"], case["Hkv"], case["ps"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    prefix_of = s["prefix_of"].tolist() if s["prefix_of"] is not None else [-1] * B
    win_len = s["win_len"].tolist() if s["win_len"] is not None else [K] * B
    parent = s["parent"].tolist() if s["parent"] is not None else [[t - 1 for t in range(K)]] * B
    out = torch.zeros((B, K, Hq, case["D"]), dtype=torch.float64, device="cuda")
    lse = torch.full((B, K, Hq), -math.inf, dtype=torch.float64, device="cuda")

    def tokens(cache, slot):
        if slot < 0 or lens[slot] == 0:
            return cache[0, 0, :0]
        ids = torch.tensor(table[slot][:-(-lens[slot] // ps)], device="cuda")
        return cache[0].index_select(0, ids).flatten(0, 1)[:lens[slot]]

    for b in range(B):
        w = win_len[b]
        seen = torch.zeros((w, w), dtype=torch.bool)
        for t in range(w):
            j = t
            while j >= 0:
                seen[t, j] = True
                j = parent[b][j]
        k, v = (torch.cat([tokens(cache, prefix_of[b]), tokens(cache, b), win[b, :w]]).double()
                for cache, win in ((s["k_cache"], s["k_win"]), (s["v_cache"], s["v_win"])))
        mask = torch.cat([torch.ones((w, k.shape[0] - w), dtype=torch.bool), seen], 1).cuda()
        for h in range(Hq):
            x = s["q"][b, :w, h].double() @ k[:, h * Hkv // Hq].T * s["scale"]
            x = x.masked_fill(~mask, -math.inf)
            lse[b, :w, h] = torch.logsumexp(x, -1)
            out[b, :w, h] = torch.softmax(x, -1) @ v[:, h * Hkv // Hq]
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------- work
def work(case):
    c = dict(case)
    row = 2 * c["Hkv"] * c["D"]  # bytes of one token's keys (or values) in one layer
    rng = np.random.default_rng(0)
    if c["op"] == "attn":
        lens = int(_lens(c["lo"], c["hi"], c["B"], rng).sum())
        wins = _lens(1, c["K"], c["B"], rng) if c["ragged"] else np.full(c["B"], c["K"])
        rows = c["B"] * c["K"] * c["Hq"]
        keys = float((wins * (c["plen"] * (c["P"] > 0) + lens / c["B"] + (wins + 1) / 2)).sum())
        return {"bytes": 2 * row * (c["P"] * c["plen"] + lens + int(wins.sum())) + 4 * rows * c["D"] + 4 * rows,
                "flops": 4.0 * c["D"] * c["Hq"] * keys}
    if c["op"] == "commit":
        n = int(_lens(1, c["K"], c["B"], rng).sum())  # a tree's accepted path is at most this long
        moved = n if not c["tree"] else (n + c["B"]) // 2
        return {"bytes": 4 * row * c["layers"] * moved + 8 * c["n_pages"], "flops": 0}
    if c["op"] == "fork":
        # about four in ten takers share a sequence with an earlier one; half a page is filled
        moved = int(0.4 * c["slots"]) * min(c["ps"], c["hi"] + 1) // 2
        return {"bytes": 4 * row * c["layers"] * moved + 8 * c["n_pages"], "flops": 0}
    live = int(c["live"] * c["n_pages"])
    moved = live * (c["n_pages"] - live) // c["n_pages"]
    return {"bytes": 4 * row * c["layers"] * c["ps"] * moved + 8 * c["n_pages"], "flops": 0}
