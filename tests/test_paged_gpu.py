"""Paged-cache calls on a GB300 against plain implementations in 64 bits:
append with norm and rotation, tree attention, the accepted path, and the
three together as a decoding step runs them."""
import math

import numpy as np
import pytest
import torch

from split_w4a16_quantized_gb300 import qmm as Q

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
BF16_HALF, F16_HALF, E4M3_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -11, 2.0 ** -4, 2.0 ** -24


@pytest.fixture(autouse=True)
def _status():
    yield
    torch.cuda.synchronize()
    assert Q.qmm_kernel_status(clear=True) == 0


def _dev(x):
    return torch.as_tensor(np.ascontiguousarray(x)).cuda()


class Problem:
    """A cache with scattered pages and NaN in every slot that holds no token.

    lens, n: cached and new tokens of each sequence; values holds them in 64
    bits, [pool][b] of [lens + n, Hkv, D], as the cache's type rounds them."""

    def __init__(self, lens, n, Hkv, D, page, dtype="bf16", layout="hnd", seed=0, spare=2,
                 width=None, k_scale=None, v_scale=None):
        rng = np.random.default_rng(seed)
        self.lens, self.n = list(lens), list(n)
        self.B, self.Hkv, self.D, self.page = len(lens), Hkv, D, page
        self.fp8 = dtype == "e4m3"
        self.scales = (k_scale or 0.0125, v_scale or 0.011) if self.fp8 else (1.0, 1.0)
        need = [-(-(a + b) // page) for a, b in zip(lens, n)]
        self.width = width or max(max(need), 1) + 1
        pages = sum(need) + spare
        ids = iter(rng.permutation(pages))
        self.table = np.full((self.B, self.width), -1, np.int32)
        for b, m in enumerate(need):
            self.table[b, :m] = [next(ids) for _ in range(m)]
        shape = (pages, Hkv, page, D) if layout == "hnd" else (pages, page, Hkv, D)
        pools, self.values = [], []
        for i in range(2):
            pool = torch.full(shape, float("nan"), dtype=torch.float32)
            view = pool if layout == "hnd" else pool.transpose(1, 2)
            vals = []
            for b in range(self.B):
                x = torch.from_numpy(rng.standard_normal((lens[b] + n[b], Hkv, D)).astype(np.float32))
                x = (x / self.scales[i]).to(E4M3).float() if self.fp8 else x.bfloat16().float()
                for s in range(lens[b] + n[b]):
                    view[self.table[b, s // page], :, s % page] = x[s]
                vals.append(x.double() * self.scales[i])
            self.values.append(vals)
            pool = pool.to(E4M3 if self.fp8 else torch.bfloat16).cuda()
            pools.append(pool if layout == "hnd" else pool.transpose(1, 2))
        self.K, self.V = pools
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.N, self.T = int(self.cu[-1]), max(max(n), 1)
        self.uniform = len(set(n)) == 1 and n[0] > 0
        self.bind()

    def bind(self):
        self.d_table, self.d_lens = _dev(self.table), _dev(np.asarray(self.lens, np.int32))
        self.cache = Q.kv_cache(self.K, self.V, self.d_table, self.d_lens, *self.scales)

    def cu_arg(self):
        return None if self.uniform else _dev(self.cu)


def _tree(rng, n, kind):
    if kind == "chain":
        return np.arange(-1, n - 1)
    if kind == "star":
        return np.where(np.arange(n) == 0, -1, 0)
    p = np.array([-1] + [int(rng.integers(max(0, i - 8), i)) for i in range(1, n)])
    if kind == "forest" and n > 2:     # several roots, and values that are no parents
        p[n // 2] = -1
        p[n - 1] = n + 3
        p[1] = 1
    return p[:n]


def _ancestors(p, i):
    out = [i]
    while 0 <= p[out[-1]] < out[-1]:
        out.append(int(p[out[-1]]))
    return out


def _attention64(pb, q, parents, scale, missing=()):
    """O in 64 bits, sum_l p_l |v_l|, and the largest scale * sum |q k| of a row:
    [N, Hq, D], the same, [N, Hq].  missing: (b, page index) without storage."""
    N, Hq, D = q.shape
    qg = Hq // pb.Hkv
    O, A, S = (torch.zeros(s, dtype=torch.float64) for s in ((N, Hq, D), (N, Hq, D), (N, Hq)))
    for b in range(pb.B):
        n, ln = pb.n[b], pb.lens[b]
        K, V = pb.values[0][b], pb.values[1][b]
        gone = torch.zeros(ln + n, dtype=torch.bool)
        for bb, pi in missing:
            if bb == b:
                gone[pi * pb.page:(pi + 1) * pb.page] = True
        for i in range(n):
            see = torch.zeros(ln + n, dtype=torch.bool)
            see[:ln] = True
            see[[ln + j for j in _ancestors(parents[pb.cu[b]:], i)]] = True
            see &= ~gone
            if not see.any():
                continue
            x = q[pb.cu[b] + i].double().view(pb.Hkv, qg, D)
            s = torch.einsum("hgd,lhd->hgl", x, K[see]) * scale
            p = torch.softmax(s, -1)
            r = pb.cu[b] + i
            O[r] = torch.einsum("hgl,lhd->hgd", p, V[see]).reshape(Hq, D)
            A[r] = torch.einsum("hgl,lhd->hgd", p, V[see].abs()).reshape(Hq, D)
            S[r] = torch.einsum("hgd,lhd->hgl", x.abs(), K[see].abs()).amax(-1).reshape(Hq) * scale
    return O, A, S


def _limit(pb, O, A, S, T, D):
    """How far O may be off, per element.  Rounding O: half a step of BF16.  The
    weights, relative to each: one rounding before the product with V (BF16, or
    F16 for an 8-bit cache), and the errors of its score s in FP32: D products
    summed and one scaling, (D + 2) 2^-24 of sum |q k|, as exp turns them into
    relative ones, twice (numerator and sum).  Sums over the positions: at most
    64 terms each side in a row before a tile's result joins the FP32 total,
    bounded by 2^-24 times the number of additions in sequence (tiles plus 64
    plus the states merged), below 2^-24 * 1024 here."""
    weight = F16_HALF if pb.fp8 else BF16_HALF
    return BF16_HALF * O.abs() + A * (weight + 2 * (D + 2) * F32_HALF * S[..., None] +
                                      1024 * F32_HALF) + 1e-30


def _run_attention(pb, q, parents, scale=0.0, stream=None, ws=None):
    N, Hq, D = q.shape
    O = torch.full((N, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    if ws is None:
        nb = Q.qmm_tree_attention_workspace_bytes(pb.cache, Hq, pb.T)
        ws = torch.full((nb // 4,), float("nan"), device="cuda")
    Q.qmm_tree_attention(pb.cache, q, O, pb.T, parents=None if parents is None else _dev(
        np.asarray(parents, np.int32)), cu=pb.cu_arg(), scale=scale, workspace=ws, stream=stream)
    return O


def _check_attention(pb, Hq, kind="tree", scale=0.0, seed=1, q_scale=2.0, missing=()):
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(q_scale * rng.standard_normal((pb.N, Hq, pb.D))).bfloat16()
    parents = np.concatenate([_tree(rng, m, "chain" if kind == "none" else kind) for m in pb.n]) \
        .astype(np.int32)
    got = _run_attention(pb, q.cuda(), None if kind == "none" else parents, scale)
    again = _run_attention(pb, q.cuda(), None if kind == "none" else parents, scale)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), again.view(torch.int16)), "not deterministic"
    O, A, S = _attention64(pb, q, parents, scale or 1 / math.sqrt(pb.D), missing)
    # (a cached value past 448 scales is E4M3's NaN, as torch's conversion forms
    # it: the outputs that see it are NaN, and no others)
    fine = torch.isfinite(O)
    assert bool((torch.isfinite(got.cpu().float()) == fine).all()), "NaN in other places"
    off = torch.where(fine, (got.cpu().double() - O).abs(), 0.0)
    lim = _limit(pb, O, A, S, pb.T, pb.D)
    bad = (off > lim).nonzero()
    assert len(bad) == 0, "%d of %d off, first %s: %g, allowed %g" % (
        len(bad), off.numel(), bad[0].tolist(), off[tuple(bad[0])], lim[tuple(bad[0])])
    return got


# ---- attention ---------------------------------------------------------------

ATTENTION = [
    # lens, n, Hq, Hkv, D, page, dtype, layout, tree
    ([0], [1], 1, 1, 64, 8, "bf16", "hnd", "none"),
    ([0], [1], 4, 1, 128, 16, "e4m3", "hnd", "tree"),
    ([1000], [1], 32, 8, 128, 16, "bf16", "hnd", "none"),
    ([63, 64, 65, 0, 127, 128, 129], [1] * 7, 8, 2, 128, 64, "bf16", "nhd", "none"),
    ([62, 63, 64, 0, 126, 1], [2] * 6, 4, 2, 64, 32, "bf16", "hnd", "tree"),
    ([5, 700, 0, 61], [8] * 4, 16, 4, 128, 16, "bf16", "nhd", "tree"),
    ([5, 700, 0, 61], [8] * 4, 16, 4, 128, 16, "e4m3", "hnd", "tree"),
    ([5, 333, 0, 61], [7, 3, 0, 9], 6, 2, 64, 8, "e4m3", "nhd", "forest"),
    ([5, 333, 0, 61], [7, 3, 0, 9], 10, 2, 128, 8, "bf16", "nhd", "forest"),
    ([100, 30], [64, 64], 8, 2, 128, 128, "bf16", "hnd", "tree"),
    ([100, 30], [33, 61], 21, 3, 128, 32, "bf16", "hnd", "star"),
    ([100, 30], [33, 61], 21, 3, 128, 32, "e4m3", "nhd", "star"),
    ([100, 30], [33, 61], 8, 1, 64, 256, "e4m3", "hnd", "tree"),
    ([77, 400], [256, 256], 8, 2, 128, 64, "bf16", "nhd", "tree"),
    ([77, 400], [256, 200], 8, 2, 64, 64, "bf16", "nhd", "none"),
    ([77, 400], [256, 200], 2, 2, 128, 64, "e4m3", "nhd", "chain"),
    ([3], [3], 64, 1, 128, 16, "bf16", "hnd", "tree"),
    ([3], [5], 64, 1, 64, 16, "e4m3", "hnd", "tree"),
    ([20000, 3, 1500], [4, 4, 4], 8, 2, 128, 64, "bf16", "hnd", "tree"),
    ([20000, 3, 1500], [20, 1, 4], 8, 2, 128, 64, "bf16", "hnd", "tree"),
    ([20000, 3, 1500], [20, 1, 4], 8, 2, 64, 16, "e4m3", "nhd", "tree"),
]


@pytest.mark.parametrize("lens,n,Hq,Hkv,D,page,dtype,layout,kind", ATTENTION,
                         ids=["%d" % i for i in range(len(ATTENTION))])
def test_attention(lens, n, Hq, Hkv, D, page, dtype, layout, kind):
    _check_attention(Problem(lens, n, Hkv, D, page, dtype, layout), Hq, kind)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 4, 9, 40])
def test_attention_many_sequences(n, dtype):
    """More sequences than threads look them up with, lengths from 0 on."""
    rng = np.random.default_rng(5)
    lens = [int(v) for v in rng.integers(0, 90, 333)]
    _check_attention(Problem(lens, [n] * 333, 1, 64, 16, dtype, seed=3), 4, "tree")


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 24])
def test_attention_leaves_missing_pages_out(n, dtype):
    pb = Problem([200, 40, 10, 0], [n] * 4, 2, 128, 16, dtype)
    pages = pb.K.shape[0]
    missing = [(0, 3), (0, 4), (1, 0), (2, 0), (3, 0)] + [(b, pi) for b in (2, 3) for pi in range(4)]
    for i, (b, pi) in enumerate(missing):
        pb.table[b, pi] = [-1, pages, 2 ** 31 - 1, -2 ** 31][i % 4]
    pb.bind()
    got = _check_attention(pb, 8, "tree", missing=missing)
    rows = got[pb.cu[2]:].cpu().float()
    assert (rows == 0).all(), "tokens that see nothing get zeros"


def test_attention_past_the_table():
    """Cached tokens up to the table's end: the drafted ones have no slots."""
    pb = Problem([64, 64], [0, 0], 2, 128, 16, width=4)
    pb.n, pb.cu, pb.N, pb.T = [3, 3], np.array([0, 3, 6], np.int32), 6, 3
    pb.uniform = True
    rng = np.random.default_rng(0)
    q = torch.from_numpy(rng.standard_normal((6, 8, 128))).bfloat16()
    got = _run_attention(pb, q.cuda(), [-1, 0, 0] * 2).cpu().double()
    pb.n = [0, 0]
    for b in range(2):
        s = torch.einsum("nhgd,lhd->nhgl", q[3 * b:3 * b + 3].double().view(3, 2, 4, 128),
                         pb.values[0][b]) / math.sqrt(128)
        want = torch.einsum("nhgl,lhd->nhgd", s.softmax(-1), pb.values[1][b]).reshape(3, 8, 128)
        assert (got[3 * b:3 * b + 3] - want).abs().max() < 2 * BF16_HALF * pb.values[1][b].abs().max()
    pb.lens = [2 ** 31 - 1, -7]          # clamped: the whole table, nothing
    pb.bind()
    got2 = _run_attention(pb, q.cuda(), [-1, 0, 0] * 2).cpu().double()
    assert torch.equal(got2[:3], got[:3])
    assert torch.isfinite(got2).all()


def test_attention_scale_extremes():
    pb = Problem([300, 20], [4, 4], 2, 128, 32)
    _check_attention(pb, 8, scale=1e-3)
    _check_attention(pb, 8, q_scale=60.0)       # one weight takes nearly all
    pb8 = Problem([300, 20], [4, 4], 2, 128, 32, "e4m3", k_scale=0.3, v_scale=30.0)
    _check_attention(pb8, 8, q_scale=1e-4)
    _check_attention(pb8, 8, q_scale=200.0, scale=1e-3)


def test_attention_other_rows_untouched_and_strided_q():
    pb = Problem([90, 17], [5, 3], 2, 128, 16)
    rng = np.random.default_rng(2)
    wide = torch.from_numpy(rng.standard_normal((12, 20, 128))).bfloat16().cuda()
    q = wide[:, 4:12]                               # a view: token stride 20 * 128
    O = torch.full((12, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(Q.qmm_tree_attention_workspace_bytes(pb.cache, 8, 5), dtype=torch.uint8,
                     device="cuda")
    par = np.concatenate([_tree(rng, 5, "tree"), _tree(rng, 3, "tree"), [0] * 4]).astype(np.int32)
    Q.qmm_tree_attention(pb.cache, q, O, 5, parents=_dev(par), cu=_dev(pb.cu), workspace=ws)
    want = _run_attention(pb, q[:8].contiguous(), par[:8])
    assert torch.equal(O[:8].view(torch.int16), want.view(torch.int16))
    assert (O[8:] == 7.0).all()


def test_attention_bad_ranges_stay_in_bounds():
    """cu is device data: values out of order or range are clamped."""
    pb = Problem([30, 30, 30], [4, 4, 4], 2, 64, 16)
    q = torch.randn((12, 4, 64), device="cuda").bfloat16()
    O = torch.zeros_like(q)
    ws = torch.empty(Q.qmm_tree_attention_workspace_bytes(pb.cache, 4, 4), dtype=torch.uint8,
                     device="cuda")
    for cu in ([0, 99, 3, 12], [-5, 4, 8, 2 ** 31 - 1], [12, 8, 4, 0], [0, 12, 12, 12]):
        Q.qmm_tree_attention(pb.cache, q, O, 4, cu=_dev(np.array(cu, np.int32)), workspace=ws)
        Q.qmm_kv_append(pb.cache, q[:, :2], q[:, :2], q[:, 2:], torch.empty_like(q[:, :2]),
                        cu=_dev(np.array(cu, np.int32)))
    torch.cuda.synchronize()


def test_attention_workspace_too_small():
    pb = Problem([30], [4], 2, 64, 16)
    q = torch.zeros((4, 4, 64), dtype=torch.bfloat16, device="cuda")
    nb = Q.qmm_tree_attention_workspace_bytes(pb.cache, 4, 4)
    for ws in (None, torch.empty(nb - 16, dtype=torch.uint8, device="cuda")):
        with pytest.raises(Q.QmmError) as e:
            Q.qmm_tree_attention(pb.cache, q, q.clone(), 4, workspace=ws)
        assert e.value.code == Q.QMM_EWORKSPACE


@pytest.mark.parametrize("n", [1, 8, 48])
def test_attention_two_streams_and_graph(n):
    pb = Problem([900, 40, 333], [n] * 3, 2, 128, 16)
    rng = np.random.default_rng(4)
    q = torch.from_numpy(rng.standard_normal((pb.N, 8, 128))).bfloat16().cuda()
    par = _dev(np.concatenate([_tree(rng, n, "tree") for _ in range(3)]).astype(np.int32))
    nb = Q.qmm_tree_attention_workspace_bytes(pb.cache, 8, n)
    want = _run_attention(pb, q, par.cpu().numpy())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):
        O = torch.zeros_like(q)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[i % 2]):
            for _ in range(20):
                Q.qmm_tree_attention(pb.cache, q, O, n, parents=par, workspace=ws)
        outs.append((O, ws))
    torch.cuda.synchronize()
    for O, _ in outs:
        assert torch.equal(O.view(torch.int16), want.view(torch.int16))
    # a graph follows the device's lens and q, not those of the capture
    O, ws = torch.zeros_like(q), torch.empty(nb, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Q.qmm_tree_attention(pb.cache, q, O, n, parents=par, workspace=ws)
    pb.d_lens.copy_(_dev(np.array([333, 20, 0], np.int32)))
    g.replay()
    torch.cuda.synchronize()
    eager = torch.zeros_like(q)
    Q.qmm_tree_attention(pb.cache, q, eager, n, parents=par, workspace=ws)
    assert torch.equal(O.view(torch.int16), eager.view(torch.int16))
    assert not torch.equal(O.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("e4m3", 128), ("bf16", 64), ("e4m3", 64)])
@pytest.mark.parametrize("rows", [15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256])
def test_attention_row_borders(rows, dtype, D):
    """One query head per KV head: as many rows as tokens, on both sides of each
    border between kernels, tiles and shared-memory layouts."""
    _check_attention(Problem([150, 0, 64], [rows, 1, rows - 1], 2, D, 32, dtype, seed=rows), 2)


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "e4m3")])
def test_attention_most_rows(D, dtype):
    """256 tokens of 64 query heads per KV head."""
    _check_attention(Problem([70], [256], 1, D, 64, dtype), 64)


def test_attention_thousands_of_sequences():
    rng = np.random.default_rng(6)
    lens = [int(v) for v in rng.integers(0, 20, 4097)]
    _check_attention(Problem(lens, [1] * 4097, 1, 64, 8, seed=4), 2, "none")
    _check_attention(Problem(lens, [3] * 4097, 1, 64, 8, "e4m3", seed=4), 8, "tree")


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [3, 12, 40, 90])
def test_attention_values_that_are_not_numbers_stay_in_their_rows(n, dtype):
    """Rows of q with infinities, NaN, zeros, the type's largest and smallest
    values: what the formula makes NaN is, and every other row is what it is
    without them, bit for bit."""
    pb = Problem([130, 5], [n, n], 2, 128, 16, dtype)
    rng = np.random.default_rng(n)
    q = torch.from_numpy(rng.standard_normal((pb.N, 8, 128))).bfloat16()
    par = np.concatenate([_tree(rng, n, "tree") for _ in range(2)]).astype(np.int32)
    clean = _run_attention(pb, q.cuda(), par).cpu()
    bad = q.clone()
    bad[0, 0, 3] = float("nan")
    bad[0, 1, 100] = float("inf")
    bad[1, 5, 0] = float("-inf")
    bad[n + 1, 7] = 0.0
    bad[n + 2, 6] = 2.0 ** -133            # BF16's smallest
    got = _run_attention(pb, bad.cuda(), par).cpu()
    touched = torch.zeros((pb.N, 8), dtype=torch.bool)
    for r, h in ((0, 0), (0, 1), (1, 5)):
        touched[r, h] = True
        assert not torch.isfinite(got[r, h].float()).any()
    for r, h in ((n + 1, 7), (n + 2, 6)):
        touched[r, h] = True
    O, A, S = _attention64(pb, torch.nan_to_num(bad, 0, 0, 0), par, 1 / math.sqrt(128))
    lim = _limit(pb, O, A, S, n, 128)
    for r, h in ((n + 1, 7), (n + 2, 6)):
        assert ((got[r, h].double() - O[r, h]).abs() <= lim[r, h]).all()
    assert torch.equal(got[~touched].view(torch.int16), clean[~touched].view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 2, 9, 40])
def test_attention_small_weights_keep_their_bits(n, dtype):
    """One key takes all but 2^-15 of the weight and has no V: the output is
    what weights of 2^-23.5 each make of the others."""
    pb = Problem([300], [n], 2, 128, 16, dtype, seed=11)
    for pool, vals in ((pb.K, pb.values[0][0]), (pb.V, pb.values[1][0])):
        if vals is pb.values[0][0]:
            vals.zero_()
            vals[0, :, 0] = 448 * pb.scales[0] if pb.fp8 else 5.625
        else:
            vals[0] = 0
        for s in range(300 + n):
            row = vals[s] / (pb.scales[0] if vals is pb.values[0][0] else pb.scales[1])
            pool[int(pb.table[0, s // 16]), :, s % 16] = row.float().to(pool.dtype).cuda()
    q = torch.zeros((n, 8, 128), dtype=torch.bfloat16)
    q[:, :, 0] = 2.90625                    # 2.90625 * 5.6 = 16.3 = 23.5 log2 units
    parents = np.arange(-1, n - 1).astype(np.int32)
    got = _run_attention(pb, q.cuda(), parents, 1.0).cpu().double()
    O, A, S = _attention64(pb, q, parents, 1.0)
    lim = _limit(pb, O, A, S, n, 128)
    assert ((got - O).abs() <= lim).all(), ((got - O).abs() / lim).max()


@pytest.mark.parametrize("how", ["kv by head", "kv by row", "padded rows"])
@pytest.mark.parametrize("n", [2, 30])
def test_attention_of_pools_with_gaps(n, how):
    """K and V woven into one allocation, and rows with space behind them."""
    pb = Problem([70, 9], [n, n], 2, 64, 16)
    want = _check_attention(pb, 8)
    P = pb.K.shape[0]
    if how == "kv by head":
        both = torch.full((P, 2, 2, 16, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        K, V = both[:, 0], both[:, 1]
    elif how == "kv by row":
        both = torch.full((P, 2, 16, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        K, V = both[..., :64], both[..., 64:]
    else:
        K, V = (torch.full((P, 2, 16, 72), float("nan"), dtype=torch.bfloat16,
                           device="cuda")[..., :64] for _ in range(2))
    K.copy_(pb.K), V.copy_(pb.V)
    pb.K, pb.V = K, V
    pb.bind()
    got = _check_attention(pb, 8)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_one_page_of_one_head_in_a_view():
    """Dimensions of one row: their strides mean nothing."""
    pb = Problem([3], [4], 1, 128, 8, spare=0, width=1)
    want = _check_attention(pb, 2)
    for strides in ((8, 0, 128, 1), (0, 24, 128, 1)):
        odd = [x.as_strided((1, 1, 8, 128), strides) for x in (pb.K, pb.V)]
        pb.cache = Q.kv_cache(odd[0], odd[1], pb.d_table, pb.d_lens)
        got = _check_attention(pb, 2)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("n", [1, 40])
def test_two_graphs_with_workspaces_of_their_own(n):
    """Captured calls replayed side by side, over and over, keep their results."""
    pbs = [Problem([700, 31], [n, n], 2, 128, 16, seed=s) for s in (1, 2)]
    rng = np.random.default_rng(3)
    par = np.concatenate([_tree(rng, n, "tree") for _ in range(2)]).astype(np.int32)
    d_par = _dev(par)
    runs = []
    for pb in pbs:
        q = torch.from_numpy(rng.standard_normal((pb.N, 8, 128))).bfloat16().cuda()
        want = _run_attention(pb, q, par)
        O = torch.zeros_like(q)
        ws = torch.empty(Q.qmm_tree_attention_workspace_bytes(pb.cache, 8, n), dtype=torch.uint8,
                         device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                Q.qmm_tree_attention(pb.cache, q, O, n, parents=d_par, workspace=ws)
        runs.append((g, O, want, torch.cuda.Stream(), q, ws))
    for _ in range(10):
        for g, _, _, st, _, _ in runs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, O, want, _, _, _ in runs:
        assert torch.equal(O.view(torch.int16), want.view(torch.int16))


def test_pools_beyond_32_bits():
    """Pages whose offsets pass 2^32 bytes and 2^31 values: append, attention and
    the accepted path reach them and nothing else."""
    B, n, Hkv, page, D = 2, 6, 8, 64, 128
    pages = 40000                                   # of 128 KB: 5.2 GB a pool
    free, _ = torch.cuda.mem_get_info()
    if free < 16 << 30:
        pytest.skip("needs 11 GB")
    small = Problem([90, 10], [n, n], Hkv, D, page, seed=8)
    K, V = (torch.empty((pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    far = np.array([[pages - 1, pages - 3], [pages - 2, 5]], np.int32)
    for pool, src in ((K, small.K), (V, small.V)):
        pool[pages - 8:] = 0
        pool[:8] = 0
        for b in range(B):
            for i in range(2):
                if small.table[b, i] >= 0:
                    pool[int(far[b, i])] = src[int(small.table[b, i])]
    rng = np.random.default_rng(9)
    x = [torch.from_numpy(rng.standard_normal((B * n, Hkv, D))).bfloat16().cuda() for _ in range(2)]
    q = torch.from_numpy(rng.standard_normal((B * n, 16, D))).bfloat16().cuda()
    par = np.concatenate([_tree(rng, n, "tree") for _ in range(B)]).astype(np.int32)
    tok = np.arange(B * n, dtype=np.int32)
    path = [0, 2, 3, 5]
    for b in range(B):                              # the chain 0, 2, 3, 5 is accepted
        for a, c in zip(path, path[1:]):
            par[b * n + c] = a
    tgt = np.full(B * n, -1, np.int32)
    for b in range(B):
        for a, c in zip(path, path[1:]):
            tgt[b * n + a] = tok[b * n + c]
    got = []
    for k, v, table in ((small.K, small.V, small.d_table[:, :2].contiguous()), (K, V, _dev(far))):
        cache = Q.kv_cache(k, v, table, small.d_lens)
        Q.qmm_kv_append(cache, None, x[0], x[1])
        O = torch.empty_like(q)
        ws = torch.empty(Q.qmm_tree_attention_workspace_bytes(cache, 16, n), dtype=torch.uint8,
                         device="cuda")
        Q.qmm_tree_attention(cache, q, O, n, parents=_dev(par), workspace=ws)
        out = [torch.empty((B, n), dtype=torch.int32, device="cuda"),
               torch.empty(B, dtype=torch.int32, device="cuda")]
        Q.qmm_tree_accept(Q.kv_caches([cache]), _dev(tok), _dev(tgt), n, out[0], out[1],
                          parents=_dev(par))
        torch.cuda.synchronize()
        assert out[1].tolist() == [4, 4] and out[0][:, :4].tolist() == [path, path]
        rows = [pool[int(table[b, s // page]), :, s % page]
                for pool in (k, v) for b in range(B)
                for s in range(small.lens[b], small.lens[b] + 4)]
        got.append((O, torch.stack(rows)))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("T", [4, 40])
def test_attention_ranges_without_tokens_and_longer_than_T(T):
    pb = Problem([20, 30], [T + 3, T], 2, 64, 16)
    q = torch.randn((pb.N, 4, 64), device="cuda").bfloat16()
    ws = torch.empty(Q.qmm_tree_attention_workspace_bytes(pb.cache, 4, T), dtype=torch.uint8,
                     device="cuda")
    O = torch.full_like(q, 7.0)
    Q.qmm_tree_attention(pb.cache, q, O, T, cu=_dev(np.zeros(3, np.int32)), workspace=ws)
    torch.cuda.synchronize()
    assert (O == 7.0).all()
    Q.qmm_tree_attention(pb.cache, q, O, T, cu=_dev(pb.cu), workspace=ws)
    want = torch.full_like(q, 7.0)          # the first T of the first sequence, a chain
    cu = np.array([0, T, T], np.int32)
    Q.qmm_tree_attention(pb.cache, q, want, T, cu=_dev(cu), workspace=ws)
    torch.cuda.synchronize()
    assert (O[T:T + 3] == 7.0).all() and not (O[T + 3:] == 7.0).any()
    assert torch.equal(O[:T].view(torch.int16), want[:T].view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,n", [(0, 3), (5, 7), (0, 20), (3, 40), (8, 200)])
def test_attention_more_tokens_than_slots(lens, n, dtype):
    """A chain that runs past the table's one page: the tokens there see what
    exists."""
    pb = Problem([lens], [8 - lens], 2, 64, 8, dtype, width=1)
    rng = np.random.default_rng(n)
    pb.n, pb.cu, pb.N, pb.T = [n], np.array([0, n], np.int32), n, n
    q = torch.from_numpy(rng.standard_normal((n, 8, 64))).bfloat16()
    pb.uniform = True
    got = [_run_attention(pb, q.cuda(), par).cpu().double()
           for par in (None, np.arange(-1, n - 1))]
    assert torch.equal(*got)
    K, V = pb.values[0][0], pb.values[1][0]
    for i in range(n):
        m = min(lens + i + 1, 8)
        s = torch.einsum("hgd,lhd->hgl", q[i].double().view(2, 4, 64), K[:m]) / 8
        want = torch.einsum("hgl,lhd->hgd", s.softmax(-1), V[:m]).reshape(8, 64)
        # O's rounding, the weights' and (64 + 2) 2^-24 of |q k| / 8 < 32 each in exp
        lim = (2 * BF16_HALF + 2 * 66 * F32_HALF * 32 + 1024 * F32_HALF) * V[:m].abs().max()
        assert (got[0][i] - want).abs().max() <= lim


def test_calls_from_several_threads():
    """Host threads with a stream and a workspace each, all kernels at once."""
    import threading
    jobs, errors = [], []
    for t, (n, dtype) in enumerate([(1, "bf16"), (8, "e4m3"), (40, "bf16"), (2, "e4m3")]):
        pb = Problem([300, 40], [n] * 2, 2, 128, 16, dtype, seed=t)
        q = torch.randn((pb.N, 8, 128), device="cuda").bfloat16()
        par = np.concatenate([np.arange(-1, n - 1)] * 2).astype(np.int32)
        want = _run_attention(pb, q, par)
        ws = torch.empty(Q.qmm_tree_attention_workspace_bytes(pb.cache, 8, n), dtype=torch.uint8,
                         device="cuda")
        jobs.append((pb, q, _dev(par), want, torch.zeros_like(q), ws, torch.cuda.Stream(), n))
    torch.cuda.synchronize()

    def work(pb, q, par, want, O, ws, stream, n):
        try:
            for _ in range(100):
                Q.qmm_tree_attention(pb.cache, q, O, n, parents=par, workspace=ws,
                                     stream=stream.cuda_stream)
            stream.synchronize()
        except Exception as e:                                  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for _, _, _, want, O, _, _, _ in jobs:
        assert torch.equal(O.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("n", [1, 12, 80])
def test_attention_without_programmatic_launch(n):
    pb = Problem([500, 3], [n] * 2, 2, 128, 16)
    q = torch.randn((pb.N, 8, 128), device="cuda").bfloat16()
    want = _run_attention(pb, q, None)
    torch.cuda.synchronize()
    Q.qmm_set_pdl(0)
    try:
        got = _run_attention(pb, q, None)
        torch.cuda.synchronize()
    finally:
        Q.qmm_set_pdl(1)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


# ---- append ---------------------------------------------------------------------

def _cos_sin(rows, dim, base=1e4):
    ang = np.arange(rows)[:, None] * base ** (-np.arange(0, dim, 2) / dim)
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float()


def _turned(x, w, cs, dim, interleaved, eps):
    """Norm and rotation in 64 bits, and the sum of the magnitudes that go in."""
    x = x.double().clone()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    mag = x.abs()
    if dim:
        c, s = cs[:, None, :dim // 2].double(), cs[:, None, dim // 2:].double()
        i = torch.arange(dim // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + dim // 2)
        u, v = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = u * c - v * s, v * c + u * s
        mag[..., a], mag[..., b] = u.abs() * c.abs() + v.abs() * s.abs(), \
            v.abs() * c.abs() + u.abs() * s.abs()
    return x, mag


# FP32 work before the rounding: the norm's sum of D squares (a tree of 8 in a
# row and log2 steps), a square root, two products and the rotation's two: under
# 32 roundings of 2^-24 relative to the magnitudes.
FP32_WORK = 32 * F32_HALF


def _near_bf16(got, want, mag):
    off = (got.cpu().double() - want).abs()
    return (off <= BF16_HALF * want.abs() + 2 * FP32_WORK * mag + 1e-38).all()


def _near_e4m3(got, want, mag):
    """got: E4M3 numbers; want: the values they stand for over the scale.  Half a
    step of what is stored, and the FP32 work (with the division)."""
    want = want.clamp(-448, 448)
    off = (got.cpu().double() - want).abs()
    return (off <= torch.maximum(E4M3_HALF * want.abs(), torch.tensor(2.0 ** -10)) +
            2 * FP32_WORK * mag).all()


APPEND = [
    # lens, n, Hq, Hkv, D, page, dtype, layout, rot, interleaved, norm, fused qkv
    ([0], [1], 1, 1, 64, 8, "bf16", "hnd", 64, False, False, False),
    ([1000], [1], 32, 8, 128, 16, "bf16", "hnd", 128, False, True, True),
    ([15, 16, 17], [1, 1, 1], 32, 8, 128, 16, "e4m3", "nhd", 128, False, True, True),
    ([15, 0, 100], [5, 40, 1], 6, 2, 128, 16, "bf16", "nhd", 64, True, True, True),
    ([15, 0, 100], [5, 0, 41], 3, 1, 64, 32, "e4m3", "hnd", 16, False, False, False),
    ([15, 0, 100], [5, 0, 41], 5, 5, 64, 8, "bf16", "hnd", 32, True, False, True),
    ([7] * 40, [3] * 40, 4, 4, 128, 64, "bf16", "hnd", 128, True, False, True),
    ([7] * 40, [3] * 40, 0, 4, 128, 64, "e4m3", "nhd", 0, False, True, True),
    ([1, 2], [700, 300], 24, 8, 64, 128, "bf16", "nhd", 48, False, True, True),
    ([1] * 300, [int(v) for v in np.random.default_rng(0).integers(0, 5, 300)], 2, 1, 128, 8,
     "bf16", "hnd", 128, False, False, False),
]


@pytest.mark.parametrize("positions", [False, True])
@pytest.mark.parametrize("lens,n,Hq,Hkv,D,page,dtype,layout,rot,inter,norm,fused", APPEND,
                         ids=["%d" % i for i in range(len(APPEND))])
def test_append(lens, n, Hq, Hkv, D, page, dtype, layout, rot, inter, norm, fused, positions):
    pb = Problem(lens, n, Hkv, D, page, dtype, layout)
    rng = np.random.default_rng(9)
    N = pb.N
    x = torch.from_numpy(rng.standard_normal((N, Hq + 2 * Hkv, D)) *
                         np.exp(rng.standard_normal((N, 1, 1)))).bfloat16()
    xd = x.cuda()
    q, k, v = (xd[:, a:b] if fused else xd[:, a:b].contiguous()
               for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    rows = max(a + b for a, b in zip(lens, n)) + 5
    cs = _cos_sin(rows, rot) if rot else None
    qw, kw = (torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).bfloat16() for _ in range(2))
    seq = np.repeat(np.arange(pb.B), n)
    at = np.arange(N) - pb.cu[seq]
    pos = np.asarray(lens)[seq] + at
    if positions:
        pos = rng.integers(0, rows, N)
    rope = Q.rope(cs.cuda() if rot else None, inter, qw.cuda() if norm else None,
                  kw.cuda() if norm else None, 1e-5)
    old = [t.view(torch.int8 if pb.fp8 else torch.int16).clone() for t in (pb.K, pb.V)]
    out = torch.full((N, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda") if Hq else None
    Q.qmm_kv_append(pb.cache, q if Hq else None, k, v, out, rope=rope,
                    positions=_dev(pos.astype(np.int32)) if positions else None, cu=pb.cu_arg())
    torch.cuda.synchronize()
    c = cs[torch.from_numpy(pos).long()] if rot else None
    if Hq:
        want, mag = _turned(x[:, :Hq], qw if norm else None, c, rot, inter, 1e-5)
        assert _near_bf16(out, want, mag)
    wk, mk = _turned(x[:, Hq:Hq + Hkv], kw if norm else None, c, rot, inter, 1e-5)
    wv = x[:, Hq + Hkv:].double()
    slot = np.asarray(lens)[seq] + at
    page_of = torch.from_numpy(pb.table[seq, slot // page]).long().cuda()
    row = torch.from_numpy(slot % page).cuda()
    for i, (pool, want, mag) in enumerate(((pb.K, wk, mk), (pb.V, wv, wv.abs()))):
        bits = pool.view(torch.int8 if pb.fp8 else torch.int16)
        got = bits[page_of, :, row].view(pool.dtype).float()
        if pb.fp8:
            sc = float(np.float32(pb.scales[i]))
            assert _near_e4m3(got, want / sc, mag / sc)
        elif i == 1:
            assert torch.equal(got.cpu().double(), want)
        else:
            assert _near_bf16(got, want, mag)
        # every other row of the pool as it was
        keep = bits.clone()
        keep[page_of, :, row] = old[i][page_of, :, row]
        assert torch.equal(keep, old[i])


def test_append_in_place_and_skipped_tokens():
    pb = Problem([10, 5], [3, 3], 2, 128, 16)
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((8, 8, 128))).bfloat16().cuda()
    cs = _cos_sin(50, 128).cuda()
    pos = np.array([10, -1, 12, 50, 6, 2 ** 31 - 1, 3, 3], np.int32)   # 1, 3 and 5: left alone
    old = pb.K.view(torch.int16).clone()
    want = torch.full((8, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    args = dict(rope=Q.rope(cs), positions=_dev(pos), cu=_dev(pb.cu))
    Q.qmm_kv_append(pb.cache, x[:, :4], x[:, 4:6], x[:, 6:], want, **args)
    torch.cuda.synchronize()
    assert (want[[1, 3, 5, 6, 7]] == 5.0).all() and (want[[0, 2, 4]] != 5.0).any()
    for b, i, kept in ((0, 0, False), (0, 1, True), (0, 2, False), (1, 0, True), (1, 1, False),
                       (1, 2, True)):
        s = pb.lens[b] + i
        at = (int(pb.table[b, s // 16]), slice(None), s % 16)
        assert torch.equal(pb.K.view(torch.int16)[at], old[at]) == kept
    y = x.clone()
    Q.qmm_kv_append(pb.cache, y[:, :4], y[:, 4:6], y[:, 6:], y[:, :4], **args)
    assert torch.equal(y[[0, 2, 4], :4], want[[0, 2, 4]])
    assert torch.equal(y[[1, 3, 5, 6, 7]], x[[1, 3, 5, 6, 7]]) and torch.equal(y[:, 4:], x[:, 4:])


def test_append_without_slots():
    """Past the table's end and on missing pages q is still rotated."""
    pb = Problem([60, 3], [0, 0], 2, 64, 16, width=4)
    pb.table[1, 0] = pb.K.shape[0]
    pb.bind()
    x = torch.randn((16, 6, 64), device="cuda").bfloat16()
    old = pb.K.view(torch.int16).clone()
    out = torch.zeros((16, 2, 64), dtype=torch.bfloat16, device="cuda")
    Q.qmm_kv_append(pb.cache, x[:, :2], x[:, 2:4], x[:, 4:], out)
    torch.cuda.synchronize()
    assert torch.equal(out, x[:, :2])
    now = pb.K.view(torch.int16)
    for s in range(60, 64):     # the last slots of sequence 0 were written, nothing else
        at = (int(pb.table[0, s // 16]), slice(None), s % 16)
        assert torch.equal(now[at], x[s - 60, 2:4].view(torch.int16))
        now[at] = old[at]
    assert torch.equal(now, old)


def test_append_e4m3_saturates_and_keeps_nan():
    pb = Problem([0], [2], 1, 64, 8, "e4m3", k_scale=0.5, v_scale=1.0)
    k = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    k[0, 0, :6] = torch.tensor([1e30, -1e30, float("inf"), float("nan"), 224.0, 0.001], device="cuda")
    Q.qmm_kv_append(pb.cache, None, k, k)
    got = pb.K[int(pb.table[0, 0]), 0, 0].float().cpu()
    assert got[:3].tolist() == [448.0, -448.0, 448.0] and math.isnan(got[3])
    assert got[4] == 448.0 and got[5] == 0.001953125


# ---- the accepted path ----------------------------------------------------------------

def _walk(tok, tgt, par):
    path = [0] if len(tok) else []
    while path:
        kids = [i for i in range(path[-1] + 1, len(tok)) if par[i] == path[-1] and
                tok[i] == tgt[path[-1]]]
        if not kids:
            break
        path.append(kids[0])
    return path


@pytest.mark.parametrize("layers", [1, 3, 70])
@pytest.mark.parametrize("lens,n,Hkv,D,page,dtype,layout", [
    ([0], [1], 1, 64, 8, "bf16", "hnd"),
    ([30, 5, 0], [9, 9, 9], 2, 128, 16, "bf16", "nhd"),
    ([30, 5, 0, 14], [9, 0, 40, 2], 2, 128, 16, "e4m3", "hnd"),
    ([30, 7], [256, 200], 3, 64, 32, "e4m3", "nhd"),
])
def test_accept(layers, lens, n, Hkv, D, page, dtype, layout):
    rng = np.random.default_rng(layers)
    pbs = [Problem(lens, n, Hkv, D, page, dtype, layout, seed=7)]
    first = pbs[0]
    for i in range(1, layers):       # other layers: the same pages, other values
        p = object.__new__(Problem)
        p.__dict__.update(first.__dict__)
        roll = lambda t: t.roll(i, 0)                                        # noqa: E731
        bits = torch.int8 if first.fp8 else torch.int16
        p.K, p.V = (torch.empty_like(t).copy_(roll(t.contiguous().view(bits)).view(t.dtype))
                    for t in (first.K, first.V))
        p.cache = Q.kv_cache(p.K, p.V, first.d_table, first.d_lens, *first.scales)
        pbs.append(p)
    pars = [_tree(rng, m, "tree") for m in n]
    # few token values, so that paths are long and siblings often agree
    toks, tgts = ([rng.integers(0, 2, m) for m in n] for _ in range(2))
    cat = lambda v: _dev(np.concatenate(v).astype(np.int32))                 # noqa: E731
    bits = torch.int8 if first.fp8 else torch.int16
    want = [[t.contiguous().view(bits).clone() for t in (p.K, p.V)] for p in pbs]
    B, T = len(n), first.T
    path = torch.full((B, T), 99, dtype=torch.int32, device="cuda")
    count, nxt, new = (torch.full((B,), 99, dtype=torch.int32, device="cuda") for _ in range(3))
    Q.qmm_tree_accept(Q.kv_caches([p.cache for p in pbs]), cat(toks), cat(tgts), T, path, count,
                      nxt, new, parents=cat(pars), cu=first.cu_arg())
    torch.cuda.synchronize()
    for b in range(B):
        w = _walk(toks[b], tgts[b], pars[b])
        assert path[b].tolist() == w + [-1] * (T - len(w))
        assert count[b] == len(w) and new[b] == lens[b] + len(w)
        assert nxt[b] == (int(tgts[b][w[-1]]) if w else -1)
        for j, i in enumerate(w):
            s, d = lens[b] + i, lens[b] + j
            for layer in want:
                for t in layer:
                    t[first.table[b, d // page], :, d % page] = \
                        t[first.table[b, s // page], :, s % page].clone()
    for p, layer in zip(pbs, want):
        for t, w in zip((p.K, p.V), layer):
            assert torch.equal(t.contiguous().view(bits), w)


def test_accept_chain_and_optional_outputs():
    pb = Problem([4, 4], [5, 5], 1, 64, 8)
    tgt = np.array([1, 2, 3, 4, 5] * 2, np.int32)
    tok = np.array([9, 1, 2, 7, 4, 9, 1, 2, 3, 4], np.int32)
    path = torch.zeros((2, 5), dtype=torch.int32, device="cuda")
    count = torch.zeros(2, dtype=torch.int32, device="cuda")
    old = pb.K.view(torch.int16).clone()
    Q.qmm_tree_accept(Q.kv_caches([pb.cache]), _dev(tok), _dev(tgt), 5, path, count)
    assert path.tolist() == [[0, 1, 2, -1, -1], [0, 1, 2, 3, 4]] and count.tolist() == [3, 5]
    assert torch.equal(pb.K.view(torch.int16), old)     # a chain's rows are in place


def test_accept_missing_pages_are_not_moved():
    pb = Problem([7, 7], [6, 6], 2, 64, 8)
    pb.table[0, 0] = -1                      # slot 7 of sequence 0; 8 .. 12 are on page 1
    pb.table[1, 1] = pb.K.shape[0]
    pb.bind()
    par = np.array([-1, 0, 0, 2, 2, 4] * 2, np.int32)
    tok = np.array([0, 5, 6, 5, 7, 8] * 2, np.int32)
    tgt = np.array([6, 0, 7, 0, 8, 1] * 2, np.int32)
    path = torch.zeros((2, 6), dtype=torch.int32, device="cuda")
    count = torch.zeros(2, dtype=torch.int32, device="cuda")
    want = pb.K.view(torch.int16).clone()
    page = int(pb.table[0, 1])
    for j, i in ((1, 2), (2, 4), (3, 5)):
        want[page, :, 7 + j - 8] = want[page, :, 7 + i - 8].clone()
    Q.qmm_tree_accept(Q.kv_caches([pb.cache]), _dev(tok), _dev(tgt), 6, path, count,
                      parents=_dev(par))
    assert path.tolist() == [[0, 2, 4, 5, -1, -1]] * 2
    assert torch.equal(pb.K.view(torch.int16), want)


# ---- together -----------------------------------------------------------------------

@pytest.mark.parametrize("dtype,graph", [("bf16", False), ("bf16", True), ("e4m3", False)])
def test_decoding_steps(dtype, graph):
    """Prefill, then steps of draft - append - attend - accept in two layers,
    against a dense history kept in 64 bits."""
    rng = np.random.default_rng(11)
    B, Hq, Hkv, D, page, T, layers, steps = 3, 8, 2, 128, 16, 6, 2, 5
    prompt = [37, 3, 80]
    cap = 160
    width = cap // page
    fp8 = dtype == "e4m3"
    scales = (0.02, 0.015) if fp8 else (1.0, 1.0)
    dt = E4M3 if fp8 else torch.bfloat16
    pages = B * width
    table = _dev(rng.permutation(pages).reshape(B, width).astype(np.int32))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    caches = []
    for _ in range(layers):
        pools = [torch.full((pages, Hkv, page, D), float("nan"), device="cuda").to(dt) for _ in "kv"]
        caches.append(Q.kv_cache(*pools, table, lens, *scales))
    group = Q.kv_caches(caches)
    cs = _cos_sin(cap + T, D)
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).bfloat16()
    rope = Q.rope(cs.cuda(), q_norm=w.cuda(), k_norm=w.cuda())

    def stored(x, i):
        x = x.float()
        return ((x / scales[i]).clamp(-448, 448).to(E4M3).double() * scales[i]) if fp8 \
            else x.bfloat16().double()

    history = [[[] for _ in range(B)] for _ in range(layers)]      # rows (k, v) kept
    N = sum(prompt)
    cu = np.concatenate([[0], np.cumsum(prompt)]).astype(np.int32)
    for la in range(layers):
        x = torch.from_numpy(rng.standard_normal((N, Hq + 2 * Hkv, D))).bfloat16()
        xd = x.cuda()
        Q.qmm_kv_append(caches[la], xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:],
                        torch.empty_like(xd[:, :Hq]), rope=rope, cu=_dev(cu))
        pos = torch.cat([torch.arange(m) for m in prompt])
        k, _ = _turned(x[:, Hq:Hq + Hkv], w, cs[pos], D, False, 1e-6)
        for b in range(B):
            for r in range(cu[b], cu[b + 1]):
                history[la][b].append((stored(k[r], 0), stored(x[r, Hq + Hkv:], 1)))
    lens.copy_(_dev(np.asarray(prompt, np.int32)))
    now = list(prompt)

    x_d = [torch.zeros((B * T, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
           for _ in range(layers)]
    out_d = [torch.zeros((B * T, Hq, D), dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
    par_d, pos_d, tok_d, tgt_d = (torch.zeros(B * T, dtype=torch.int32, device="cuda")
                                  for _ in range(4))
    ws = torch.empty(Q.qmm_tree_attention_workspace_bytes(caches[0], Hq, T), dtype=torch.uint8,
                     device="cuda")
    path = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    count, nxt, new = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))

    def step():
        for la in range(layers):
            x = x_d[la]
            Q.qmm_kv_append(caches[la], x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], x[:, :Hq],
                            rope=rope, positions=pos_d)
            Q.qmm_tree_attention(caches[la], x[:, :Hq], out_d[la], T, parents=par_d, workspace=ws)
        Q.qmm_tree_accept(group, tok_d, tgt_d, T, path, count, nxt, new, parents=par_d)
        lens.copy_(new)

    g = None
    for s in range(steps):
        pars = [_tree(rng, T, "tree") for _ in range(B)]
        toks, tgts = (rng.integers(0, 2, (B, T)) for _ in range(2))
        depth = [[len(_ancestors(p, i)) - 1 for i in range(T)] for p in pars]
        pos = np.array([[now[b] + d for d in depth[b]] for b in range(B)]).reshape(-1)
        xs = [torch.from_numpy(rng.standard_normal((B * T, Hq + 2 * Hkv, D))).bfloat16()
              for _ in range(layers)]
        if graph and g is None:
            before = lens.clone()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            assert torch.equal(before, lens)
        for la in range(layers):
            x_d[la].copy_(xs[la])
        par_d.copy_(_dev(np.concatenate(pars).astype(np.int32)))
        pos_d.copy_(_dev(pos.astype(np.int32)))
        tok_d.copy_(_dev(toks.reshape(-1).astype(np.int32)))
        tgt_d.copy_(_dev(tgts.reshape(-1).astype(np.int32)))
        g.replay() if g is not None else step()
        torch.cuda.synchronize()
        walks = [_walk(toks[b], tgts[b], pars[b]) for b in range(B)]
        for la in range(layers):
            c = cs[torch.from_numpy(pos).long()]
            q, _ = _turned(xs[la][:, :Hq], w, c, D, False, 1e-6)
            k, _ = _turned(xs[la][:, Hq:Hq + Hkv], w, c, D, False, 1e-6)
            q = q.float().bfloat16().double()
            got = out_d[la].cpu().double()
            for b in range(B):
                new_rows = [(stored(k[b * T + i], 0), stored(xs[la][b * T + i, Hq + Hkv:], 1))
                            for i in range(T)]
                for i in range(T):
                    rows = history[la][b] + [new_rows[j] for j in _ancestors(pars[b], i)]
                    K, V = (torch.stack([r[z] for r in rows]) for z in range(2))
                    sc = torch.einsum("hgd,lhd->hgl", q[b * T + i].view(Hkv, -1, D), K) / math.sqrt(D)
                    p = sc.softmax(-1)
                    o = torch.einsum("hgl,lhd->hgd", p, V).reshape(Hq, D)
                    a = torch.einsum("hgl,lhd->hgd", p, V.abs()).reshape(Hq, D)
                    # a value at a rounding border may fall to its other side in
                    # q, in k or in the weights: one whole step of each instead
                    # of half (E4M3 keys: a score moves by 2^-3 of |q k| / sqrt(D)
                    # for at most a few of them)
                    lim = BF16_HALF * o.abs() + a * (0.03 if not fp8 else 0.06)
                    assert ((got[b * T + i] - o).abs() <= lim).all(), (s, la, b, i)
                history[la][b] += [new_rows[i] for i in walks[b]]
        for b in range(B):
            now[b] += len(walks[b])
            assert path[b].tolist() == walks[b] + [-1] * (T - len(walks[b]))
        assert lens.tolist() == now
