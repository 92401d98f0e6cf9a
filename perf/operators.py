"""Timed cases of the paged-cache operators: append with rotation, attention of
drafted trees over the cache, and the commit of an accepted path.

listed() and draw() describe cases as plain dicts, prepare() builds what a
decoding program holds before the call, run() makes one pass: in elementary
torch operations in 32 bits, or, with `own` set, through the framework's entry
points.  exact() gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

ROPE_BASE = 1.0e6
EPS = 1.0e-6


# ---- cases -----------------------------------------------------------------

def _append(name, B, T, lmin, lmax, Hq=32, Hkv=8, D=128, page=16, dtype="bf16", layout="hnd",
            ragged=False, tree=False, rot=None, interleaved=False, norm=True):
    return {"name": name, "op": "append", "B": B, "T": T, "lmin": lmin, "lmax": lmax, "Hq": Hq,
            "Hkv": Hkv, "D": D, "page": page, "dtype": dtype, "layout": layout, "ragged": ragged,
            "tree": tree, "rot": D if rot is None else rot, "interleaved": interleaved,
            "norm": norm}


def _attend(name, B, T, lmin, lmax, Hq=32, Hkv=8, D=128, page=16, dtype="bf16", layout="hnd",
            ragged=False, chain=False):
    return {"name": name, "op": "attend", "B": B, "T": T, "lmin": lmin, "lmax": lmax, "Hq": Hq,
            "Hkv": Hkv, "D": D, "page": page, "dtype": dtype, "layout": layout, "ragged": ragged,
            "chain": chain}


def _accept(name, B, T, lmin, lmax, layers, Hkv=8, D=128, page=16, dtype="bf16", layout="hnd",
            ragged=False):
    return {"name": name, "op": "accept", "B": B, "T": T, "lmin": lmin, "lmax": lmax, "Hq": 4 * Hkv,
            "Hkv": Hkv, "D": D, "page": page, "dtype": dtype, "layout": layout, "ragged": ragged,
            "layers": layers}


def listed():
    return [
        # one token of one sequence: the call between two projections, latency alone
        _append("append_decode_b1", 1, 1, 1000, 1000),
        # a batch's drafted trees before they are verified, 8-bit cache
        _append("append_verify_b32_t8_e4m3", 32, 8, 200, 9000, page=32, dtype="e4m3", tree=True),
        # a ragged prefill chunk, half of each 64-wide head rotated in adjacent pairs, no norm
        _append("append_ragged_d64", 7, 700, 1, 3000, Hq=24, Hkv=8, D=64, page=64, layout="nhd",
                ragged=True, rot=32, interleaved=True, norm=False),
        # a long prefill
        _append("append_prefill_16k", 2, 8192, 1, 1, page=64),
        # one user decoding over a short history
        _attend("attend_decode_b1", 1, 1, 1000, 1000),
        # a small batch's drafted trees: 32 query rows a KV head
        _attend("attend_verify_b8_t8", 8, 8, 1500, 4000),
        # a serving batch's decode step, histories from 1024 to 8192
        _attend("attend_decode_b32", 32, 1, 1024, 8192, page=64, chain=True),
        # wide trees: 256 query rows a KV head, where the products cost as much as the bytes
        _attend("attend_tree_b16_t64", 16, 64, 8000, 8000, page=32),
        # drafted trees over an 8-bit cache with tokens before heads in a page
        _attend("attend_tree_b32_t16_e4m3", 32, 16, 500, 16000, page=64, dtype="e4m3", layout="nhd"),
        # histories of very different lengths, trees of different sizes, 64-wide heads
        _attend("attend_ragged_b64_d64", 64, 5, 60, 32000, Hq=64, Hkv=8, D=64, page=32, ragged=True),
        # one user's accepted path committed in every layer
        _accept("accept_b1_t8", 1, 8, 700, 700, 36),
        # a batch's accepted paths, trees of different sizes
        _accept("accept_b64_t16", 64, 16, 10, 100, 36, ragged=True),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "accept"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    qg = rng.choice([1, 2, 3, 4, 4, 5, 8])
    more = dict(D=D, Hkv=Hkv, page=rng.choice([16, 16, 32, 64, 128]),
                dtype=rng.choice(["bf16", "bf16", "e4m3"]), layout=rng.choice(["hnd", "nhd"]),
                ragged=rng.random() < 0.4)
    lo = _log(rng, 1, 8000)
    if op == "append":
        B = _log(rng, 1, 48)
        T = _log(rng, 1, max(2, 12000 // B))
        return _without_name(_append("", B, T, lo, lo + _log(rng, 1, 4000), Hq=Hkv * qg,
                                     tree=T <= 64 and rng.random() < 0.5,
                                     rot=rng.choice([D, D, D // 2, 16]),
                                     interleaved=rng.random() < 0.3, norm=rng.random() < 0.5,
                                     **more))
    if op == "attend":
        B = _log(rng, 1, 48)
        T = rng.choice([1, 1, 2, 3, 4, 6, 8, 12, 16, 27, 33, 48, 64])
        hi = min(lo + _log(rng, 1, 8000), max(lo, 400000 // B))
        lo = min(lo, hi)
        return _without_name(_attend("", B, T, lo, hi, Hq=Hkv * qg, chain=rng.random() < 0.3,
                                     **more))
    B = _log(rng, 1, 48)
    lo = min(lo, 4000 // B + 1)
    return _without_name(_accept("", B, rng.choice([2, 3, 5, 8, 16, 24, 40, 64]), lo,
                                 lo + rng.randrange(1, 40), rng.choice([1, 2, 12, 28, 36]), **more))


def _without_name(c):
    del c["name"]
    return c


# ---- sizes of a case (the same for every seed, up to the order of the sequences) ----

def _lens(c):
    """Cached tokens and new tokens of each sequence."""
    B, lo, hi = c["B"], c["lmin"], c["lmax"]
    at = np.arange(B) / (B - 1) if B > 1 else np.ones(1)
    lens = np.round(lo * (hi / lo) ** at).astype(np.int64)
    n = np.full(B, c["T"], np.int64)
    if c["ragged"]:
        n = 1 + (np.arange(B) * 5 + 2) % B * (c["T"] - 1) // max(1, B - 1)
    return lens, n


def _accepted(n):
    """Accepted nodes of a tree of n nodes: up to half of them, at most 6."""
    return np.minimum((n + 1) // 2, 6)


def work(c):
    lens, n = _lens(c)
    e = 1 if c["dtype"] == "e4m3" else 2
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    N = int(n.sum())
    if c["op"] == "append":
        return {"bytes": N * ((2 * Hq + 2 * Hkv) * D * 2 + 2 * Hkv * D * e + c["rot"] * 4),
                "flops": N * (Hq + Hkv) * (3 * c["rot"] + (4 * D if c["norm"] else 0))}
    if c["op"] == "attend":
        keys = int((lens + n).sum())
        return {"bytes": 2 * keys * Hkv * D * e + 2 * N * Hq * D * 2,
                "flops": 4 * Hq * D * int(((lens + n) * n).sum())}
    moved = int((_accepted(n) - 1).sum())
    return {"bytes": 2 * moved * c["layers"] * 2 * Hkv * D * e + 16 * N, "flops": 0}


# ---- inputs ------------------------------------------------------------------

def _tree(rng, n):
    """Parents of a drafted tree: node 0 is the last sampled token, each other
    node hangs below one of the eight before it."""
    parents = np.full(n, -1, np.int64)
    if n > 1:
        i = np.arange(1, n)
        parents[1:] = i - 1 - (rng.random(n - 1) * np.minimum(i, 8)).astype(np.int64)
    return parents


def _depth(parents):
    depth = np.zeros(len(parents), np.int64)
    for i in range(1, len(parents)):
        depth[i] = depth[parents[i]] + 1
    return depth


def _accept_tree(rng, n):
    """A tree, its drafted tokens and the model's choice after each node, such
    that a path of _accepted(n) nodes is accepted.  The path's nodes lie past
    the slots they move to, so that a second pass finds the same sources."""
    a = int(_accepted(np.asarray(n)))
    path = np.concatenate([[0], a + np.sort(rng.choice(n - a, a - 1, replace=False))]).astype(int) \
        if a > 1 else np.zeros(1, int)
    parents = _tree(rng, n)
    parents[path[1:]] = path[:-1]
    targets = rng.integers(1000, 150000, n)
    tokens = rng.integers(1000, 150000, n)
    off = 1 + rng.integers(0, 900, n)
    tokens[1:] = targets[parents[1:]] + off[1:]
    tokens[path[1:]] = targets[path[:-1]]
    return parents, tokens, targets


def _pool(gen, shape, c, scale):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if c["dtype"] == "e4m3":
        return (x / scale).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return x.to(torch.bfloat16)


def prepare(c, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, T, Hq, Hkv, D, page = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    lens, n = _lens(c)
    order = rng.permutation(B)
    lens, n = lens[order], n[order]
    N, layers = int(n.sum()), c.get("layers", 1)
    # pages of each sequence, scattered over the pool
    need = -(-(lens + n) // page)
    pages = int(need.sum()) + 3
    width = int(need.max())
    ids = rng.permutation(pages)[:int(need.sum())]
    table = np.zeros((B, width), np.int32)
    table[np.arange(width)[None] < need[:, None]] = ids
    k_scale, v_scale = (0.0125, 0.011) if c["dtype"] == "e4m3" else (1.0, 1.0)
    shape = (layers, pages, Hkv, page, D) if c["layout"] == "hnd" else (layers, pages, page, Hkv, D)
    K, V = _pool(gen, shape, c, k_scale), _pool(gen, shape, c, v_scale)
    if c["layout"] == "nhd":
        K, V = K.transpose(2, 3), V.transpose(2, 3)
    cu = np.concatenate([[0], np.cumsum(n)])
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731
    seq = np.repeat(np.arange(B), n)
    at = np.arange(N) - cu[seq]
    s = {"case": c, "K": K, "V": V, "table": dev(table), "lens": dev(lens), "cu": dev(cu),
         "seq": dev(seq).long(), "at": dev(at).long(), "N": N, "k_scale": k_scale,
         "v_scale": v_scale, "parents": None}
    if c["op"] == "append":
        Dq, Dk = Hq * D, Hkv * D
        qkv = torch.randn((N, Dq + 2 * Dk), generator=gen, device="cuda").to(torch.bfloat16)
        s["q"] = qkv[:, :Dq].view(N, Hq, D)
        s["k"] = qkv[:, Dq:Dq + Dk].view(N, Hkv, D)
        s["v"] = qkv[:, Dq + Dk:].view(N, Hkv, D)
        pos = lens[seq] + at
        if c["tree"]:
            pos = lens[seq] + np.concatenate([_depth(_tree(rng, m)) for m in n])
        s["positions"] = dev(pos)
        # the program's own table of cosines and sines
        inv = ROPE_BASE ** (-np.arange(0, c["rot"], 2) / c["rot"])
        ang = np.arange(int((lens + n).max()) + 1)[:, None] * inv
        s["cos_sin"] = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float().cuda()
        w = lambda: (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(torch.bfloat16)  # noqa: E731
        s["q_norm"], s["k_norm"] = (w(), w()) if c["norm"] else (None, None)
        s["out"] = torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "attend":
        s["q"] = (2 * torch.randn((N, Hq, D), generator=gen, device="cuda")).to(torch.bfloat16)
        if not c["chain"]:
            s["parents"] = dev(np.concatenate([_tree(rng, m) for m in n]))
        s["out"] = torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda")
    else:
        trees = [_accept_tree(rng, int(m)) for m in n]
        s["parents"], s["tokens"], s["targets"] = (dev(np.concatenate(v)) for v in zip(*trees))
        s["path"] = torch.empty((B, T), dtype=torch.int32, device="cuda")
        s["count"], s["next"], s["new_lens"] = (torch.empty(B, dtype=torch.int32, device="cuda")
                                                for _ in range(3))
    if own:
        _prepare_own(s)
    return s


# ---- the framework's calls -----------------------------------------------------

def _prepare_own(s):
    from split_w4a16_quantized_gb300 import qmm as Q
    c = s["case"]
    s["Q"] = Q
    s["caches"] = [Q.kv_cache(K, V, s["table"], s["lens"], s["k_scale"], s["v_scale"])
                   for K, V in zip(s["K"], s["V"])]
    s["cu_arg"] = s["cu"] if c["ragged"] else None
    if c["op"] == "append":
        s["rope"] = Q.rope(s["cos_sin"], interleaved=c["interleaved"], q_norm=s["q_norm"],
                           k_norm=s["k_norm"], eps=EPS)
    elif c["op"] == "attend":
        nb = Q.qmm_tree_attention_workspace_bytes(s["caches"][0], c["Hq"], c["T"])
        s["ws"] = torch.empty(nb, dtype=torch.uint8, device="cuda")
    else:
        s["group"] = Q.kv_caches(s["caches"])


def _run_own(s):
    c, Q = s["case"], s["Q"]
    if c["op"] == "append":
        Q.qmm_kv_append(s["caches"][0], s["q"], s["k"], s["v"], s["out"], rope=s["rope"],
                        positions=s["positions"], cu=s["cu_arg"])
        return {"q": s["out"], "K": s["K"], "V": s["V"]}
    if c["op"] == "attend":
        Q.qmm_tree_attention(s["caches"][0], s["q"], s["out"], c["T"], parents=s["parents"],
                             cu=s["cu_arg"], workspace=s["ws"])
        return s["out"]
    Q.qmm_tree_accept(s["group"], s["tokens"], s["targets"], c["T"], s["path"], s["count"],
                      s["next"], s["new_lens"], parents=s["parents"], cu=s["cu_arg"])
    return {"path": s["path"], "count": s["count"], "next": s["next"], "lens": s["new_lens"],
            "K": s["K"], "V": s["V"]}


# ---- the plain form ---------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"append": _run_append, "attend": _run_attend, "accept": _run_accept}[s["case"]["op"]](s)


def _normed(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(x, cos, sin, c):
    r = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _stored(x, scale, like):
    if like.dtype == torch.bfloat16:
        return x.to(torch.bfloat16)
    return (x / scale).clamp(-448, 448).to(like.dtype)


def _bytes(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _run_append(s):
    c = s["case"]
    cs = s["cos_sin"][s["positions"].long()]
    cos, sin = cs[:, None, :c["rot"] // 2], cs[:, None, c["rot"] // 2:]
    q = _rotated(_normed(s["q"], s["q_norm"]), cos, sin, c)
    k = _rotated(_normed(s["k"], s["k_norm"]), cos, sin, c)
    slot = s["lens"].long()[s["seq"]] + s["at"]
    page = s["table"].long()[s["seq"], slot // c["page"]]
    row = slot % c["page"]
    K, V = s["K"][0], s["V"][0]
    _bytes(K)[page, :, row] = _bytes(_stored(k, s["k_scale"], K))
    _bytes(V)[page, :, row] = _bytes(_stored(s["v"].float(), s["v_scale"], V))
    s["out"].copy_(q)
    return {"q": s["out"], "K": s["K"], "V": s["V"]}


def _padded(s, x, fill):
    """[B, T, ...] from one row per token, with `fill` behind each sequence's last."""
    c = s["case"]
    out = torch.full((c["B"], c["T"]) + tuple(x.shape[1:]), fill, dtype=x.dtype, device=x.device)
    out[s["seq"], s["at"]] = x
    return out


def _ancestors(s):
    """[B, T, T]: whether node j is node i itself or one of its ancestors.  With
    P the matrix of parents, the sum of its powers is the inverse of I - P."""
    c = s["case"]
    B, T = c["B"], c["T"]
    if s["parents"] is None:
        return torch.ones((T, T), dtype=torch.bool, device="cuda").tril().expand(B, T, T)
    par = _padded(s, s["parents"].long(), -1)
    P = (par[:, :, None] == torch.arange(T, device="cuda")).float()
    eye = torch.eye(T, device="cuda").expand(B, T, T)
    return torch.linalg.solve_triangular(eye - P, eye, upper=False, unitriangular=True) > 0.5


def _dense(pool, s, scale):
    """The pages of every sequence in order: [B, Hkv, L, D] in 32 bits."""
    c = s["case"]
    x = _bytes(pool)[s["table"].long()]
    x = x.view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else x
    return (x.float() * scale).transpose(1, 2).reshape(c["B"], c["Hkv"], -1, c["D"])


def _run_attend(s):
    c = s["case"]
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    K, V = _dense(s["K"][0], s, s["k_scale"]), _dense(s["V"][0], s, s["v_scale"])
    L = K.shape[2]
    q = _padded(s, s["q"].float(), 0.0).view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    S = torch.matmul(q.reshape(B, Hkv, -1, D), K.transpose(2, 3)) / math.sqrt(D)
    node = torch.arange(L, device="cuda") - s["lens"].long()[:, None]          # [B, L]
    anc = _ancestors(s).gather(2, node.clamp(0, T - 1)[:, None].expand(B, T, L))
    see = (node < 0)[:, None] | (anc & ((node >= 0) & (node < T))[:, None])    # [B, T, L]
    S = S.view(B, Hkv, Hq // Hkv, T, L).masked_fill(~see[:, None, None], -math.inf)
    p = torch.exp(S - S.amax(-1, keepdim=True))
    o = torch.matmul(p.view(B, Hkv, -1, L), V).view(B, Hkv, Hq // Hkv, T, D)
    o = o / p.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D)
    s["out"].copy_(o[s["seq"], s["at"]])
    return s["out"]


def _run_accept(s):
    c = s["case"]
    B, T = c["B"], c["T"]
    par = _padded(s, s["parents"].long(), -1)
    tok, tgt = _padded(s, s["tokens"].long(), -1), _padded(s, s["targets"].long(), -1)
    # a node its parent's target names, and no sibling before it
    match = (par >= 0) & (tok == tgt.gather(1, par.clamp(min=0)))
    before = torch.ones((T, T), dtype=torch.bool, device="cuda").tril(-1)
    twin = (par[:, :, None] == par[:, None]) & match[:, None] & before
    ok = match & ~twin.any(-1)
    ok[:, 0] = True
    taken = ~(_ancestors(s) & ~ok[:, None]).any(-1)
    taken &= _padded(s, torch.ones_like(s["seq"], dtype=torch.bool), False) & ((par >= 0) | (
        torch.arange(T, device="cuda") == 0))
    count = taken.sum(-1)
    path = torch.where(taken, torch.arange(T, device="cuda"), T).sort(-1).values
    last = path.gather(1, (count - 1)[:, None])
    s["path"].copy_(torch.where(path < T, path, -1))
    s["count"].copy_(count)
    s["next"].copy_(tgt.gather(1, last)[:, 0])
    s["new_lens"].copy_(s["lens"] + count)
    # rows of the path to the front of the drafted slots (the rest onto themselves)
    first = s["lens"].long()[:, None]
    j = torch.arange(T, device="cuda").expand(B, T)
    j = torch.where(path < T, j, 0)
    src, dst = first + torch.where(path < T, path, 0), first + j
    b = torch.arange(B, device="cuda")[:, None]
    ps, pd = (s["table"].long()[b, x // c["page"]] for x in (src, dst))
    rs, rd = src % c["page"], dst % c["page"]
    K, V = _bytes(s["K"]).transpose(2, 3), _bytes(s["V"]).transpose(2, 3)
    K[:, pd, rd] = K[:, ps, rs]
    V[:, pd, rd] = V[:, ps, rs]
    return {"path": s["path"], "count": s["count"], "next": s["next"], "lens": s["new_lens"],
            "K": s["K"], "V": s["V"]}


# ---- the definitions in 64 bits ---------------------------------------------------

def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    if c["op"] == "append":
        return _exact_append(s, c, lens, cu)
    if c["op"] == "attend":
        return _exact_attend(s, c, lens, cu)
    return _exact_accept(s, c, lens, cu)


def _e4m3(x):
    """The E4M3 value nearest to x, ties to the even mantissa, in 64 bits."""
    x = x.clamp(-448.0, 448.0)
    e = torch.frexp(x).exponent.double() - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(s, c, lens, cu):
    r = c["rot"]
    pos = s["positions"].long()

    def turn(x, w):
        x = x.double().clone()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
        cs = s["cos_sin"].double()[pos].unsqueeze(1)
        z = torch.complex(cs[..., :r // 2], cs[..., r // 2:])
        i = torch.arange(r // 2, device="cuda")
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
        y = torch.complex(x[..., a], x[..., b]) * z
        x[..., a], x[..., b] = y.real, y.imag
        return x

    K, V = s["K"].double(), s["V"].double()
    k, v = turn(s["k"], s["k_norm"]) / s["k_scale"], s["v"].double() / s["v_scale"]
    if c["dtype"] == "e4m3":
        k, v = _e4m3(k), _e4m3(v)
    table = s["table"].long()
    for b in range(c["B"]):
        slot = lens[b] + torch.arange(cu[b + 1] - cu[b], device="cuda")
        at = (0, table[b, torch.div(slot, c["page"], rounding_mode="floor")], slice(None),
              slot % c["page"])
        K[at], V[at] = k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]
    return {"q": turn(s["q"], s["q_norm"]), "K": K, "V": V}


def _exact_attend(s, c, lens, cu):
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    par = s["parents"].tolist() if s["parents"] is not None else None
    qg = c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        n, ln = cu[b + 1] - cu[b], lens[b]
        see = torch.zeros((n, ln + n), dtype=torch.bool)
        see[:, :ln] = True
        for i in range(n):
            j = i
            while j >= 0:
                see[i, ln + j] = True
                j = (par[cu[b] + j] if par is not None else j - 1)
        see = see.cuda()
        slot = torch.arange(ln + n, device="cuda")
        page, row = s["table"][b].long()[slot // c["page"]], slot % c["page"]
        for h in range(c["Hkv"]):
            K = s["K"][0, :, h].double()[page, row] * s["k_scale"]
            V = s["V"][0, :, h].double()[page, row] * s["v_scale"]
            q = s["q"][cu[b]:cu[b + 1], h * qg:(h + 1) * qg].double()
            x = torch.einsum("ngd,ld->ngl", q, K) * c["D"] ** -0.5
            x = x.masked_fill(~see[:, None], -math.inf)
            out[cu[b]:cu[b + 1], h * qg:(h + 1) * qg] = torch.einsum("ngl,ld->ngd", x.softmax(-1), V)
    return out


def _exact_accept(s, c, lens, cu):
    par, tok, tgt = s["parents"].tolist(), s["tokens"].tolist(), s["targets"].tolist()
    K, V, table = _bytes(s["K"]).clone(), _bytes(s["V"]).clone(), s["table"].tolist()
    paths, nxt = [], []
    for b in range(c["B"]):
        o, n = cu[b], cu[b + 1] - cu[b]
        path = [0]
        while True:
            kids = [i for i in range(1, n) if par[o + i] == path[-1] and
                    tok[o + i] == tgt[o + path[-1]]]
            if not kids:
                break
            path.append(kids[0])
        nxt.append(tgt[o + path[-1]])
        for j, i in enumerate(path):
            a, d = lens[b] + i, lens[b] + j
            for X in (K, V):
                X[:, table[b][d // c["page"]], :, d % c["page"]] = \
                    X[:, table[b][a // c["page"]], :, a % c["page"]].clone()
        paths.append(path + [-1] * (c["T"] - len(path)))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    count = [sum(i >= 0 for i in p) for p in paths]
    return {"path": i32(paths), "count": i32(count), "next": i32(nxt),
            "lens": i32([x + y for x, y in zip(lens, count)]), "K": K.view(s["K"].dtype),
            "V": V.view(s["V"].dtype)}
