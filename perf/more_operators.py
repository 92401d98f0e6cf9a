"""Timed cases of the paged cache's long-context operators: attention of a batch
whose sequences share long prefixes, attention that adds up the weight each slot
receives, eviction by that weight, and append with positions of several axes.

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

def _prefix(name, B, T, plen, lmin, lmax, groups=1, Hq=32, Hkv=8, D=128, page=16, dtype="bf16",
            layout="hnd", ragged=False, tree=False):
    """groups: prefixes that the batch's sequences share, of plen tokens down to a
    quarter of it; lmin, lmax: each sequence's own tokens behind its prefix."""
    return {"name": name, "op": "prefix", "B": B, "T": T, "plen": plen, "lmin": lmin, "lmax": lmax,
            "groups": groups, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "dtype": dtype,
            "layout": layout, "ragged": ragged, "tree": tree}


def _scored(name, B, T, lmin, lmax, decay=1.0, Hq=32, Hkv=8, D=128, page=16, dtype="bf16",
            layout="hnd", ragged=False):
    return {"name": name, "op": "scored", "B": B, "T": T, "lmin": lmin, "lmax": lmax,
            "decay": decay, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "dtype": dtype,
            "layout": layout, "ragged": ragged}


def _evict(name, B, lmin, lmax, keep, sinks, recent, layers, Hkv=8, D=128, page=16, dtype="bf16",
           layout="hnd"):
    return {"name": name, "op": "evict", "B": B, "T": 1, "lmin": lmin, "lmax": lmax, "keep": keep,
            "sinks": sinks, "recent": recent, "layers": layers, "Hq": 4 * Hkv, "Hkv": Hkv, "D": D,
            "page": page, "dtype": dtype, "layout": layout, "ragged": False}


def _axes(name, B, T, lmin, lmax, axes=3, alternating=False, Hq=32, Hkv=8, D=128, page=16,
          dtype="bf16", layout="hnd", ragged=False, rot=None, interleaved=False, norm=True):
    """axes: positions of a token; alternating: neighbouring pairs turn by
    different axes, else each axis has a section of the pairs."""
    return {"name": name, "op": "axes", "B": B, "T": T, "lmin": lmin, "lmax": lmax, "axes": axes,
            "alternating": alternating, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "dtype": dtype,
            "layout": layout, "ragged": ragged, "rot": D if rot is None else rot,
            "interleaved": interleaved, "norm": norm}


def listed():
    return [
        # four users of one short system prompt: latency
        _prefix("prefix_decode_b4_p500", 4, 1, 500, 20, 60),
        # a serving batch's decode step behind one long document
        _prefix("prefix_decode_b64_p8k", 64, 1, 8192, 100, 1000, page=64),
        # drafted trees of a batch behind a long 8-bit prefix, trees of different sizes
        _prefix("prefix_verify_b24_t8_e4m3", 24, 8, 16000, 100, 900, page=32, dtype="e4m3",
                layout="nhd", ragged=True, tree=True),
        # several prompts' groups of very different lengths, 64-wide heads
        _prefix("prefix_groups_b48_d64", 48, 4, 20000, 30, 3000, groups=5, Hq=64, D=64, page=32),
        # one user's decode step while the weights are added up: latency
        _scored("scored_decode_b1", 1, 1, 1000, 1000),
        # a serving batch's decode step, histories from 1024 to 8192
        _scored("scored_decode_b32", 32, 1, 1024, 8192, page=64),
        # an 8-bit cache, 64-wide heads in groups of 8, old weights fading
        _scored("scored_decode_b64_d64_e4m3", 64, 1, 300, 12000, decay=0.98, Hq=64, D=64, page=32,
                dtype="e4m3", layout="nhd"),
        # the last tokens of long prompts score the prompts before a first eviction
        _scored("scored_window_b8_t32", 8, 32, 2000, 16000, decay=0.0, page=32, ragged=True),
        # one user's cache goes back to its budget in every layer
        _evict("evict_b1_36layers", 1, 1151, 1151, 1024, 4, 256, 36),
        # a batch's prompts cut to the budget
        _evict("evict_b16_12layers", 16, 2500, 7000, 2048, 4, 512, 12, page=32, layout="nhd"),
        # one image's patches behind a few words: a small prompt's call
        _axes("axes_image_b1", 1, 300, 1, 1),
        # a batch of video prompts, ragged, pairs of the axes in turn, into an 8-bit cache
        _axes("axes_video_b6_e4m3", 6, 3000, 1, 2000, alternating=True, page=64, dtype="e4m3",
              ragged=True),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "scored", "scored", "evict", "axes"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8])
    qg = rng.choice([1, 2, 3, 4, 4, 5, 8])
    kind = dict(D=D, Hkv=Hkv, page=rng.choice([16, 16, 32, 64, 128]),
                dtype=rng.choice(["bf16", "bf16", "e4m3"]), layout=rng.choice(["hnd", "nhd"]))
    more = dict(kind, Hq=Hkv * qg, ragged=rng.random() < 0.4)
    lo = _log(rng, 1, 4000)
    if op == "prefix":
        B = _log(rng, 1, 64)
        T = rng.choice([1, 1, 1, 2, 3, 4, 6, 8, 16])
        plen = min(_log(rng, 1, 20000), 4000000 // (B * T))
        hi = min(lo + _log(rng, 1, 3000), max(lo, 90000 // B))
        return _without_name(_prefix("", B, T, plen, min(lo, hi), hi,
                                     groups=rng.randrange(1, min(B, 6) + 1),
                                     tree=rng.random() < 0.6, **more))
    if op == "scored":
        B = _log(rng, 1, 48)
        T = rng.choice([1, 1, 1, 1, 2, 3, 4, 7, 16, 32, 64])
        hi = min(lo + _log(rng, 1, 8000), max(lo, 200000 // B))
        hi = min(hi, 2000000 // (B * T) + 1)
        return _without_name(_scored("", B, T, min(lo, hi), hi,
                                     decay=rng.choice([0.0, 0.5, 0.98, 1.0]), **more))
    if op == "evict":
        B, layers = _log(rng, 1, 16), rng.choice([1, 2, 5, 12])
        hi = min(lo + _log(rng, 1, 8000), 300000 // (B * layers) + 2)
        lo = min(lo, hi)
        keep = _log(rng, 1, hi)
        sinks = rng.randrange(0, min(keep, 8) + 1)
        return _without_name(_evict("", B, lo, hi, keep, sinks,
                                    int((keep - sinks) * rng.choice([0.0, 0.1, 0.25, 0.5, 1.0])),
                                    layers, **kind))
    B = _log(rng, 1, 32)
    T = _log(rng, 1, max(2, 9000 // B))
    return _without_name(_axes("", B, T, lo, lo + _log(rng, 1, 4000), axes=rng.choice([2, 3, 3, 4]),
                               alternating=rng.random() < 0.5, rot=rng.choice([D, D, D // 2, 16]),
                               interleaved=rng.random() < 0.3, norm=rng.random() < 0.5, **more))


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


def _groups(c):
    """Tokens of each prefix, and the first sequence of each group (and B)."""
    G = c["groups"]
    at = np.arange(G) / (G - 1) if G > 1 else np.zeros(1)
    plens = np.maximum(1, np.round(c["plen"] * 0.25 ** at)).astype(np.int64)
    return plens, (np.arange(G + 1) * c["B"]) // G


def work(c):
    lens, n = _lens(c)
    e = 1 if c["dtype"] == "e4m3" else 2
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    N = int(n.sum())
    row = 2 * Hkv * D * e          # bytes of a position's K and V
    if c["op"] == "prefix":
        plens, first = _groups(c)
        tokens = np.add.reduceat(n, first[:-1])
        pairs = int(((lens + n) * n).sum() + (plens * tokens).sum())
        return {"bytes": int((lens + n).sum() + plens.sum()) * row + 2 * N * Hq * D * 2,
                "flops": 4 * Hq * D * pairs}
    if c["op"] == "scored":
        keys = int((lens + n).sum())
        return {"bytes": keys * row + 2 * N * Hq * D * 2 + keys * Hkv * 4 +
                (int(lens.sum()) * Hkv * 4 if c["decay"] else 0),
                "flops": 4 * Hq * D * int(((lens + n) * n).sum())}
    if c["op"] == "evict":
        keep, s, r = c["keep"], c["sinks"], c["recent"]
        cut = lens[lens > keep]
        # rows that move: the recent ones, and the part of the others' choice that
        # lies behind the slots it goes to (expected)
        moved = (r + (keep - s - r) * (cut - keep) / (cut - s - r)).sum() if len(cut) else 0.0
        # (weights by columns of a head)
        ints = int(lens.sum() + 2 * np.minimum(lens, keep).sum()) * 4
        return {"bytes": c["layers"] * (2 * float(moved) * row + Hkv * ints), "flops": 0}
    return {"bytes": N * ((2 * Hq + 2 * Hkv) * D * 2 + row + c["axes"] * 4 + c["rot"] * 4),
            "flops": N * (Hq + Hkv) * (3 * c["rot"] + (4 * D if c["norm"] else 0))}


# ---- inputs ------------------------------------------------------------------

def _tree(rng, n):
    """Parents of a drafted tree: node 0 is the last sampled token, each other
    node hangs below one of the eight before it."""
    parents = np.full(n, -1, np.int64)
    if n > 1:
        i = np.arange(1, n)
        parents[1:] = i - 1 - (rng.random(n - 1) * np.minimum(i, 8)).astype(np.int64)
    return parents


def _pool(gen, shape, c, scale):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if c["dtype"] == "e4m3":
        return (x / scale).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return x.to(torch.bfloat16)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _tables(rng, need, spare):
    """Page tables over one pool, pages scattered: a row for each entry of need."""
    pages = int(need.sum()) + spare
    ids = rng.permutation(pages)[:int(need.sum())]
    table = np.zeros((len(need), int(need.max())), np.int32)
    table[np.arange(table.shape[1])[None] < need[:, None]] = ids
    return table, pages


def _image_positions(rng, n, axes):
    """Positions [axes, n] of a prompt: words, whose axes agree, then patches in
    rows and columns, frame after frame."""
    words = max(1, int(n * rng.uniform(0.05, 0.3)))
    i = np.arange(max(0, n - words))
    w = int(rng.integers(4, 40))
    h = int(rng.integers(4, 40))
    grid = [i // (w * h), i // w % h, i % w, i // 7]
    if axes == 2:
        grid = grid[1:3]
    pos = np.empty((axes, n), np.int64)
    for a in range(axes):
        pos[a, :words] = np.arange(words)
        pos[a, words:] = words + grid[a]
    return pos


def _axis_of_pair(c):
    """Axis that each of the rot / 2 pairs turns by."""
    half, A = c["rot"] // 2, c["axes"]
    j = np.arange(half)
    if c["alternating"]:
        return j % A
    # the first axis has half of an equal share's pairs less than the others
    lead = max(1, half // A * 3 // 4)
    return np.where(j < lead, 0, np.minimum(A - 1, 1 + (j - lead) * (A - 1) // max(1, half - lead)))


def prepare(c, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, Hq, Hkv, D, page = c["B"], c["Hq"], c["Hkv"], c["D"], c["page"]
    lens, n = _lens(c)
    order = rng.permutation(B)
    lens, n = lens[order], n[order]
    if c["op"] == "evict":
        n = np.zeros_like(n)
    N, layers = int(n.sum()), c.get("layers", 1)
    need = -(-(lens + n) // page)
    if c["op"] == "prefix":
        plens, first = _groups(c)
        need = np.concatenate([need, -(-plens // page)])
    table, pages = _tables(rng, need, 3)
    k_scale, v_scale = (0.0125, 0.011) if c["dtype"] == "e4m3" else (1.0, 1.0)
    shape = (layers, pages, Hkv, page, D) if c["layout"] == "hnd" else (layers, pages, page, Hkv, D)
    K, V = _pool(gen, shape, c, k_scale), _pool(gen, shape, c, v_scale)
    if c["layout"] == "nhd":
        K, V = K.transpose(2, 3), V.transpose(2, 3)
    cu = np.concatenate([[0], np.cumsum(n)])
    seq = np.repeat(np.arange(B), n)
    at = np.arange(N) - cu[seq]
    s = {"case": c, "K": K, "V": V, "table": _dev(table[:B]), "lens": _dev(lens), "cu": _dev(cu),
         "seq": _dev(seq).long(), "at": _dev(at).long(), "N": N, "k_scale": k_scale,
         "v_scale": v_scale, "parents": None}
    if c["op"] == "axes":
        Dq, Dk = Hq * D, Hkv * D
        qkv = torch.randn((N, Dq + 2 * Dk), generator=gen, device="cuda").to(torch.bfloat16)
        s["q"] = qkv[:, :Dq].view(N, Hq, D)
        s["k"] = qkv[:, Dq:Dq + Dk].view(N, Hkv, D)
        s["v"] = qkv[:, Dq + Dk:].view(N, Hkv, D)
        pos = np.concatenate([ln + _image_positions(rng, int(m), c["axes"])
                              for ln, m in zip(lens, n)], 1)
        s["positions"] = _dev(pos)
        s["axis_of_pair"] = [int(a) for a in _axis_of_pair(c)]
        s["axis"] = torch.tensor(s["axis_of_pair"], device="cuda")
        # the program's own table of cosines and sines
        inv = ROPE_BASE ** (-np.arange(0, c["rot"], 2) / c["rot"])
        ang = np.arange(int(pos.max()) + 1)[:, None] * inv
        s["cos_sin"] = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float().cuda()
        w = lambda: (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(torch.bfloat16)  # noqa: E731
        s["q_norm"], s["k_norm"] = (w(), w()) if c["norm"] else (None, None)
        s["out"] = torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "evict":
        # weights differ by orders of magnitude, and some slots have none
        S = s["table"].shape[1] * page
        mass = torch.exp(1.5 * torch.randn((layers, B, Hkv, S), generator=gen, device="cuda"))
        mass *= torch.rand(mass.shape, generator=gen, device="cuda") > 0.05
        s["mass"], s["mass_out"] = mass, torch.zeros_like(mass)
        s["kept"] = torch.empty((layers, B, Hkv, c["keep"]), dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
    else:
        s["q"] = (2 * torch.randn((N, Hq, D), generator=gen, device="cuda")).to(torch.bfloat16)
        s["out"] = torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda")
        if c["op"] == "scored":
            S = s["table"].shape[1] * page
            s["mass"] = torch.exp(torch.randn((B, Hkv, S), generator=gen, device="cuda"))
        else:
            if c["tree"]:
                s["parents"] = _dev(np.concatenate([_tree(rng, int(m)) for m in n]))
            s["ptable"], s["plens"], s["first"] = _dev(table[B:]), _dev(plens), _dev(first)
            group = np.repeat(np.arange(c["groups"]), np.diff(first))
            s["group"] = _dev(group).long()
            s["in_group"] = _dev(np.arange(B) - first[group]).long()
            s["widest"] = int(np.diff(first).max())
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
    nb = 0
    if c["op"] == "prefix":
        s["prefix"] = Q.prefix(s["ptable"], s["plens"], s["first"])
        nb = Q.qmm_prefix_attention_workspace_bytes(s["caches"][0], c["Hq"], s["N"], c["T"])
    elif c["op"] == "scored":
        nb = Q.qmm_scored_attention_workspace_bytes(s["caches"][0], c["Hq"], c["T"])
    elif c["op"] == "evict":
        s["group"] = Q.kv_caches(s["caches"])
    else:
        s["rope"] = Q.rope(s["cos_sin"], interleaved=c["interleaved"], q_norm=s["q_norm"],
                           k_norm=s["k_norm"], eps=EPS)
        s["axes"] = Q.rope_axes(s["axis_of_pair"])
    s["ws"] = torch.empty(nb, dtype=torch.uint8, device="cuda")


def _run_own(s):
    c, Q = s["case"], s["Q"]
    if c["op"] == "prefix":
        Q.qmm_prefix_attention(s["caches"][0], s["prefix"], s["q"], s["out"], c["T"],
                               parents=s["parents"], cu=s["cu_arg"], workspace=s["ws"])
        return s["out"]
    if c["op"] == "scored":
        Q.qmm_scored_attention(s["caches"][0], s["q"], s["out"], c["T"], s["mass"],
                               decay=c["decay"], cu=s["cu_arg"], workspace=s["ws"])
        return {"out": s["out"], "mass": s["mass"]}
    if c["op"] == "evict":
        Q.qmm_kv_evict(s["group"], s["mass"], c["keep"], s["kept"], s["new_lens"],
                       sinks=c["sinks"], recent=c["recent"], mass_out=s["mass_out"])
        return {"kept": s["kept"], "lens": s["new_lens"], "mass": s["mass_out"], "K": s["K"],
                "V": s["V"]}
    Q.qmm_kv_append_axes(s["caches"][0], s["q"], s["k"], s["v"], s["positions"], s["axes"],
                         s["rope"], q_out=s["out"], cu=s["cu_arg"])
    return {"q": s["out"], "K": s["K"], "V": s["V"]}


# ---- the plain form ---------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"prefix": _run_prefix, "scored": _run_scored, "evict": _run_evict,
            "axes": _run_axes}[s["case"]["op"]](s)


def _bytes(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


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


def _dense(pool, table, scale):
    """The pages of a table's rows in order: [rows, Hkv, L, D] in 32 bits."""
    x = _bytes(pool)[table.long()]
    x = x.view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else x
    x = (x.float() * scale).transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[4])


def _queries(s):
    """q as [B, Hkv, QG, T, D] in 32 bits, scaled."""
    c = s["case"]
    q = _padded(s, s["q"].float(), 0.0).view(c["B"], c["T"], c["Hkv"], -1, c["D"])
    return q.permute(0, 2, 3, 1, 4) / math.sqrt(c["D"])


def _own_scores(s, q, K):
    """Scores of a sequence's own slots, -inf where a token does not see them:
    [B, Hkv, QG, T, L]."""
    c = s["case"]
    B, T, L = c["B"], c["T"], K.shape[2]
    S = torch.matmul(q.flatten(2, 3), K.transpose(2, 3)).view(q.shape[:4] + (L,))
    node = torch.arange(L, device="cuda") - s["lens"].long()[:, None]          # [B, L]
    anc = _ancestors(s).gather(2, node.clamp(0, T - 1)[:, None].expand(B, T, L))
    see = (node < 0)[:, None] | (anc & ((node >= 0) & (node < T))[:, None])    # [B, T, L]
    return S.masked_fill(~see[:, None, None], -math.inf)


def _tokens_out(s, o):
    """[B, Hkv, QG, T, D] to the rows of s["out"]."""
    c = s["case"]
    o = o.permute(0, 3, 1, 2, 4).reshape(c["B"], c["T"], c["Hq"], c["D"])
    s["out"].copy_(o[s["seq"], s["at"]])


def _run_prefix(s):
    c = s["case"]
    B, T, Hkv, D, G, W = c["B"], c["T"], c["Hkv"], c["D"], c["groups"], s["widest"]
    q = _queries(s)
    K, V = (_dense(s[x][0], s["table"], s[y]) for x, y in (("K", "k_scale"), ("V", "v_scale")))
    PK, PV = (_dense(s[x][0], s["ptable"], s[y]) for x, y in (("K", "k_scale"), ("V", "v_scale")))
    S = _own_scores(s, q, K)
    # all rows of a group against its prefix at once
    qg = torch.zeros((G, W) + q.shape[1:], device="cuda")
    qg[s["group"], s["in_group"]] = q
    qg = qg.transpose(1, 2)                                           # [G, Hkv, W, QG, T, D]
    P = PK.shape[2]
    SP = torch.matmul(qg.reshape(G, Hkv, -1, D), PK.transpose(2, 3))
    gone = torch.arange(P, device="cuda") >= s["plens"].long()[:, None]
    SP = SP.masked_fill(gone[:, None, None], -math.inf).view(qg.shape[:5] + (P,))
    top = torch.maximum(S.amax(-1), SP.transpose(1, 2)[s["group"], s["in_group"]].amax(-1))
    p = torch.exp(S - top[..., None])
    tg = torch.zeros((G, W) + top.shape[1:], device="cuda")
    tg[s["group"], s["in_group"]] = top
    pp = torch.exp(SP - tg.transpose(1, 2)[..., None])
    op = torch.matmul(pp.flatten(2, 4), PV).view(qg.shape).transpose(1, 2)[s["group"], s["in_group"]]
    sums = p.sum(-1) + pp.sum(-1).transpose(1, 2)[s["group"], s["in_group"]]
    o = torch.matmul(p.flatten(2, 3), V).view(q.shape) + op
    _tokens_out(s, o / sums[..., None])
    return s["out"]


def _run_scored(s):
    c = s["case"]
    q = _queries(s)
    K, V = (_dense(s[x][0], s["table"], s[y]) for x, y in (("K", "k_scale"), ("V", "v_scale")))
    S = _own_scores(s, q, K)
    p = torch.exp(S - S.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    _tokens_out(s, torch.matmul(p.flatten(2, 3), V).view(q.shape))
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    real = torch.arange(c["T"], device="cuda") < n[:, None]                    # [B, T]
    w = (p * real[:, None, None, :, None]).sum((2, 3))                         # [B, Hkv, L]
    slot = torch.arange(w.shape[-1], device="cuda")
    lens = s["lens"].long()[:, None, None]
    old = torch.where(slot < lens, s["mass"] * c["decay"], 0.0)
    s["mass"].copy_(torch.where(slot < lens + n[:, None, None], old + w, s["mass"]))
    return {"out": s["out"], "mass": s["mass"]}


def _run_evict(s):
    c = s["case"]
    keep, sinks, recent = c["keep"], c["sinks"], c["recent"]
    mass = s["mass"]                                                 # [layers, B, Hkv, S]
    S = mass.shape[-1]
    slot = torch.arange(S, device="cuda")
    lens = s["lens"].long()[:, None, None]                           # [B, 1, 1]
    new = lens.clamp(max=keep)
    # the sinks, the recent ones and the heaviest of the others, lowest slot first
    forced = (slot < sinks) | ((slot >= lens - recent) & (slot < lens))
    order = torch.where(forced, math.inf, torch.where(slot < lens, mass, -1.0))
    order = order.sort(dim=-1, descending=True, stable=True).indices
    chosen = torch.zeros(mass.shape, dtype=torch.bool, device="cuda")
    chosen.scatter_(-1, order[..., :keep], True)
    chosen &= slot < lens
    # slots below `line` are filled in place: each evicted one takes the next
    # chosen one at or behind the line; the recent ones follow in order
    line = new - torch.where(lens > keep, recent, 0)
    hole = ~chosen & (slot < line)
    late = chosen & (slot >= line) & (slot < lens - torch.where(lens > keep, recent, 0))
    rank = torch.where(hole, hole.cumsum(-1) - 1, 0)
    late_slots = torch.where(late, slot, S).sort(dim=-1).values
    kept = torch.where(hole, late_slots.gather(-1, rank), slot.expand_as(mass))
    kept = torch.where(slot >= line, slot + lens - new, kept)[..., :keep]
    live = slot[:min(keep, S)] < new
    kept = torch.where(live, kept, -1)
    if kept.shape[-1] < keep:
        kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[-1]), value=-1)
    s["kept"].copy_(kept)
    s["new_lens"].copy_(new[:, 0, 0])
    src = kept[..., :S].clamp(min=0)
    moved = mass.gather(-1, src)
    to = s["mass_out"][..., :src.shape[-1]]
    to.copy_(torch.where(live, moved, to))
    # rows by (sequence, head, slot)
    b = torch.arange(c["B"], device="cuda")[:, None, None]
    h = torch.arange(c["Hkv"], device="cuda")[None, :, None]
    lay = torch.arange(c["layers"], device="cuda")[:, None, None, None]
    j = slot[:src.shape[-1]].expand_as(src)
    src, dst = torch.where(live, src, j), j
    ps, pd = (s["table"].long()[b, x // c["page"]] for x in (src, dst))
    rs, rd = src % c["page"], dst % c["page"]
    at, h, b = live & (src != dst), h.expand_as(src), b.expand_as(src)
    lay = lay.expand_as(src)
    for pool in (s["K"], s["V"]):
        x = _bytes(pool)
        x[lay[at], pd[at], h[at], rd[at]] = x[lay[at], ps[at], h[at], rs[at]]
    return {"kept": s["kept"], "lens": s["new_lens"], "mass": s["mass_out"], "K": s["K"],
            "V": s["V"]}


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


def _run_axes(s):
    c = s["case"]
    half = c["rot"] // 2
    pos = s["positions"].long().t()[:, s["axis"]]                    # [N, rot / 2]
    pair = torch.arange(half, device="cuda")
    cos, sin = s["cos_sin"][pos, pair][:, None], s["cos_sin"][pos, pair + half][:, None]
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


# ---- the definitions in 64 bits ---------------------------------------------------

def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    if c["op"] == "evict":
        return _exact_evict(s, c, lens)
    if c["op"] == "axes":
        return _exact_axes(s, c, lens, cu)
    return _exact_attention(s, c, lens, cu)


def _exact_attention(s, c, lens, cu):
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if c["op"] == "scored" else None
    par = s["parents"].tolist() if s["parents"] is not None else None
    qg, page = c["Hq"] // c["Hkv"], c["page"]
    group = s["group"].tolist() if c["op"] == "prefix" else None
    for b in range(c["B"]):
        n, ln = cu[b + 1] - cu[b], lens[b]
        sees = np.zeros((n, ln + n), bool)
        sees[:, :ln] = True
        for i in range(n):
            j = i
            while j >= 0:
                sees[i, ln + j] = True
                j = (par[cu[b] + j] if par is not None else j - 1)
        slot = torch.arange(ln + n, device="cuda")
        pages, rows = s["table"][b].long()[slot // page], slot % page
        if group is not None:
            g = group[b]
            before = torch.arange(int(s["plens"][g]), device="cuda")
            pages = torch.cat([s["ptable"][g].long()[before // page], pages])
            rows = torch.cat([before % page, rows])
            sees = np.concatenate([np.ones((n, len(before)), bool), sees], 1)
        sees = torch.from_numpy(sees).cuda()
        for h in range(c["Hkv"]):
            K = s["K"][0, :, h].double()[pages, rows] * s["k_scale"]
            V = s["V"][0, :, h].double()[pages, rows] * s["v_scale"]
            q = s["q"][cu[b]:cu[b + 1], h * qg:(h + 1) * qg].double()
            x = torch.einsum("ngd,ld->ngl", q, K) * c["D"] ** -0.5
            w = x.masked_fill(~sees[:, None], -math.inf).softmax(-1)
            out[cu[b]:cu[b + 1], h * qg:(h + 1) * qg] = torch.einsum("ngl,ld->ngd", w, V)
            if mass is not None:
                mass[b, h, :ln] *= c["decay"]
                mass[b, h, ln:ln + n] = 0.0
                mass[b, h, :ln + n] += w.sum((0, 1))
    return out if mass is None else {"out": out, "mass": mass}


def _exact_evict(s, c, lens):
    keep, sinks, recent, page = c["keep"], c["sinks"], c["recent"], c["page"]
    K, V = _bytes(s["K"]).cpu(), _bytes(s["V"]).cpu()
    mass, table = s["mass"].double().cpu().numpy(), s["table"].cpu().numpy().astype(np.int64)
    kept = np.full(s["kept"].shape, -1, np.int64)
    after = np.zeros_like(mass)
    for layer in range(c["layers"]):
        for b, ln in enumerate(lens):
            m = min(ln, keep)
            for h in range(c["Hkv"]):
                w = mass[layer, b, h, :ln]
                where = list(range(m))
                if ln > keep:
                    middle = np.arange(sinks, ln - recent)
                    best = middle[np.argsort(-w[middle], kind="stable")][:keep - sinks - recent]
                    best = set(best.tolist())
                    line = keep - recent
                    late = sorted(i for i in best if i >= line)
                    for i in range(sinks, line):
                        if i not in best:
                            where[i] = late.pop(0)
                    where[line:] = range(ln - recent, ln)
                where = np.asarray(where, np.int64)
                kept[layer, b, h, :m] = where
                after[layer, b, h, :m] = w[where]
                dst = np.nonzero(where != np.arange(m))[0]
                src = where[dst]
                for X in (K, V):
                    rows = X[layer, table[b, src // page], h, src % page].clone()
                    X[layer, table[b, dst // page], h, dst % page] = rows
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32)  # noqa: E731
    return {"kept": i32(kept), "lens": i32([min(x, keep) for x in lens]),
            "mass": torch.from_numpy(after), "K": K.view(s["K"].dtype), "V": V.view(s["V"].dtype)}


def _e4m3(x):
    """The E4M3 value nearest to x, ties to the even mantissa, in 64 bits."""
    x = x.clamp(-448.0, 448.0)
    e = torch.frexp(x).exponent.double() - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_axes(s, c, lens, cu):
    r = c["rot"]

    def turn(x, w):
        x = x.double().clone()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
        for j, a in enumerate(s["axis_of_pair"]):
            cs = s["cos_sin"].double()[s["positions"][a].long()]
            z = torch.complex(cs[:, j], cs[:, j + r // 2])[:, None]
            one, two = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + r // 2)
            y = torch.complex(x[..., one], x[..., two]) * z
            x[..., one], x[..., two] = y.real, y.imag
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
