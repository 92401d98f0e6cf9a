"""The paged cache's long-context calls on a GB300 against plain implementations in 64
bits: shared prefixes, weights by slot, eviction, positions of several axes, and the
calls together as a decoding program runs them."""
import math

import numpy as np
import pytest
import torch

from split_w4a16_quantized_gb300 import qmm as Q
from test_paged_gpu import BF16_HALF, F16_HALF, F32_HALF, Problem, _ancestors, _cos_sin, _dev, \
    _near_bf16, _near_e4m3, _tree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    yield
    torch.cuda.synchronize()
    assert Q.qmm_kernel_status(clear=True) == 0


def _same(a, b):
    return torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32),
                       b.view(torch.int16 if b.element_size() == 2 else torch.int32))


def _within(got, want, lim):
    """(A cached value past 448 scales is E4M3's NaN, as torch's conversion forms it:
    what sees it is NaN, and nothing else is.)"""
    fine = torch.isfinite(want)
    assert bool((torch.isfinite(got) == fine).all()), "NaN in other places"
    off = (got.double() - want).abs()
    bad = (fine & ~(off <= lim)).nonzero()
    if len(bad):
        at = tuple(bad[0])
        raise AssertionError("%d of %d off, first %s: %g, allowed %g (of %g)" % (
            len(bad), off.numel(), bad[0].tolist(), off[at], lim[at], want[at]))


# ---- shared prefixes -----------------------------------------------------------------

class Shared:
    """Sequences behind prefixes over one pool: plens[g] tokens shared by the sequences
    first[g] .. first[g + 1] - 1."""

    def __init__(self, plens, first, lens, n, Hkv, D, page, dtype="bf16", layout="hnd", seed=0,
                 **kw):
        self.pb = pb = Problem(list(lens) + list(plens), list(n) + [0] * len(plens), Hkv, D, page,
                               dtype, layout, seed, **kw)
        self.B, self.G, self.first, self.plens = len(lens), len(plens), list(first), list(plens)
        self.lens, self.n = list(lens), list(n)
        self.cu = pb.cu[:self.B + 1].copy()
        self.N, self.T = int(self.cu[-1]), max(max(n), 1)
        self.uniform = len(set(n)) == 1 and n[0] > 0
        self.bind()

    def bind(self):
        pb = self.pb
        self.d_lens = _dev(np.asarray(self.lens, np.int32))
        self.d_plens = _dev(np.asarray(self.plens, np.int32))
        self.d_first = _dev(np.asarray(self.first, np.int32))
        self.cache = Q.kv_cache(pb.K, pb.V, _dev(pb.table[:self.B]), self.d_lens, *pb.scales)
        self.prefix = Q.prefix(_dev(pb.table[self.B:]), self.d_plens, self.d_first)

    def cu_arg(self):
        return None if self.uniform else _dev(self.cu)

    def group(self, b):
        return next((g for g in range(self.G) if self.first[g] <= b < self.first[g + 1]), None)

    def rows(self, b, missing=()):
        """Keys and values of sequence b in 64 bits: the prefix's, then its own; which of
        them have pages; how many are the prefix's."""
        pb, g = self.pb, self.group(b)
        parts = ([] if g is None else [self.B + g]) + [b]
        K, V = (torch.cat([pb.values[i][x] for x in parts]) for i in range(2))
        there = torch.ones(len(K), dtype=torch.bool)
        before = 0 if g is None else len(pb.values[0][self.B + g])
        for x, pi in missing:
            if x in parts:
                off = before if x == b else 0
                end = min((pi + 1) * pb.page, len(pb.values[0][x]))
                there[off + pi * pb.page:off + end] = False
        return K, V, there, before


def _prefix64(sh, q, parents, scale, missing=()):
    N, Hq, D = q.shape
    Hkv = sh.pb.Hkv
    O, A, S = (torch.zeros(s, dtype=torch.float64) for s in ((N, Hq, D), (N, Hq, D), (N, Hq)))
    for b in range(sh.B):
        K, V, there, before = sh.rows(b, missing)
        for i in range(sh.n[b]):
            see = torch.zeros(len(K), dtype=torch.bool)
            see[:before + sh.lens[b]] = True
            see[[before + sh.lens[b] + j for j in _ancestors(parents[sh.cu[b]:], i)]] = True
            see &= there
            if not see.any():
                continue
            r = sh.cu[b] + i
            x = q[r].double().view(Hkv, -1, D)
            s = torch.einsum("hgd,lhd->hgl", x, K[see]) * scale
            p = torch.softmax(s, -1)
            O[r] = torch.einsum("hgl,lhd->hgd", p, V[see]).reshape(Hq, D)
            A[r] = torch.einsum("hgl,lhd->hgd", p, V[see].abs()).reshape(Hq, D)
            S[r] = torch.einsum("hgd,lhd->hgl", x.abs(), K[see].abs()).amax(-1).reshape(Hq) * scale
    return O, A, S


def _o_limit(fp8, O, A, S, D):
    """How far O may be off, per element: half a step of BF16 for the output; of the
    weights, one rounding before the product with V (BF16, or F16 for an 8-bit cache)
    and what (D + 2) 2^-24 of sum |q k| makes of an exp, twice (numerator and sum);
    sums over the positions, 2^-24 times the additions in sequence, below 1024."""
    weight = F16_HALF if fp8 else BF16_HALF
    return BF16_HALF * O.abs() + A * (weight + 2 * (D + 2) * F32_HALF * S[..., None] +
                                      1024 * F32_HALF) + 1e-30


def _run_prefix(sh, q, parents, scale=0.0, stream=None, ws=None, O=None):
    N, Hq, D = q.shape
    O = torch.full((N, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda") if O is None else O
    if ws is None:
        nb = Q.qmm_prefix_attention_workspace_bytes(sh.cache, Hq, N, sh.T)
        ws = torch.full((nb // 4,), float("nan"), device="cuda")
    Q.qmm_prefix_attention(sh.cache, sh.prefix, q, O, sh.T,
                           parents=None if parents is None else _dev(np.asarray(parents, np.int32)),
                           cu=sh.cu_arg(), scale=scale, workspace=ws, stream=stream)
    return O


def _check_prefix(sh, Hq, kind="tree", scale=0.0, seed=1, q_scale=2.0, missing=()):
    rng = np.random.default_rng(seed)
    D = sh.pb.D
    q = torch.from_numpy(q_scale * rng.standard_normal((sh.N, Hq, D))).bfloat16()
    parents = np.concatenate([_tree(rng, m, kind) for m in sh.n]).astype(np.int32)
    given = None if kind == "chain" else parents
    got, again = (_run_prefix(sh, q.cuda(), given, scale) for _ in range(2))
    torch.cuda.synchronize()
    assert _same(got, again), "not deterministic"
    O, A, S = _prefix64(sh, q, parents, scale or 1 / math.sqrt(D), missing)
    _within(got.cpu(), O, _o_limit(sh.pb.fp8, O, A, S, D))
    return got


PREFIX = [
    # plens, first, lens, n, Hq, Hkv, D, page, dtype, layout, tree
    ([1], [0, 1], [0], [1], 1, 1, 64, 8, "bf16", "hnd", "chain"),
    ([64], [0, 2], [0, 1], [1, 1], 4, 1, 128, 16, "e4m3", "hnd", "tree"),
    ([500], [0, 4], [20, 30, 40, 60], [1] * 4, 32, 8, 128, 16, "bf16", "hnd", "chain"),
    ([63, 64, 65], [0, 2, 3, 7], [0, 5, 64, 63, 127, 128, 129], [1] * 7, 8, 2, 128, 64, "bf16",
     "nhd", "chain"),
    ([1000, 7], [0, 5, 9], [5, 70, 0, 61, 3, 3, 400, 9, 1], [8] * 9, 16, 4, 128, 16, "bf16", "nhd",
     "tree"),
    ([1000, 7], [0, 5, 9], [5, 70, 0, 61, 3, 3, 400, 9, 1], [8] * 9, 16, 4, 128, 16, "e4m3", "hnd",
     "tree"),
    # ranges of different sizes, none among them; sequences of no prefix on both ends
    ([333, 90], [1, 3, 6], [5, 333, 0, 61, 2, 9, 40], [7, 3, 0, 9, 1, 0, 5], 6, 2, 64, 8, "e4m3",
     "nhd", "forest"),
    ([333, 90], [1, 3, 6], [5, 333, 0, 61, 2, 9, 40], [7, 3, 0, 9, 1, 0, 5], 10, 2, 128, 8, "bf16",
     "nhd", "forest"),
    # a prefix of no tokens, one of no sequences
    ([0, 200, 100], [0, 2, 2, 4], [5, 6, 7, 0], [3] * 4, 8, 2, 64, 32, "bf16", "hnd", "tree"),
    # more rows than an item holds, on both sides of its border
    ([700], [0, 8], [3, 9, 1, 0, 2, 5, 7, 130], [4] * 8, 8, 2, 128, 16, "bf16", "hnd", "tree"),
    ([700], [0, 9], [3, 9, 1, 0, 2, 5, 7, 130, 4], [4] * 9, 7, 1, 64, 16, "e4m3", "nhd", "tree"),
    ([4000], [0, 40], list(range(40)), [1] * 40, 16, 2, 128, 64, "bf16", "nhd", "chain"),
    ([4000], [0, 3], [100, 30, 0], [33, 61, 256], 21, 3, 128, 32, "bf16", "hnd", "star"),
    ([2500], [0, 2], [100, 30], [200, 256], 8, 1, 64, 128, "e4m3", "hnd", "tree"),
    ([300], [0, 2], [3, 0], [3, 3], 64, 1, 128, 16, "bf16", "hnd", "tree"),
]


@pytest.mark.parametrize("plens,first,lens,n,Hq,Hkv,D,page,dtype,layout,kind", PREFIX,
                         ids=["%d" % i for i in range(len(PREFIX))])
def test_prefix(plens, first, lens, n, Hq, Hkv, D, page, dtype, layout, kind):
    _check_prefix(Shared(plens, first, lens, n, Hkv, D, page, dtype, layout), Hq, kind)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 5])
def test_prefix_many_sequences_and_groups(n, dtype):
    """More entries than threads look them up with; a group of each length from 0 on."""
    rng = np.random.default_rng(5)
    lens = [int(v) for v in rng.integers(0, 90, 300)]
    first = [0] + sorted(int(v) for v in rng.integers(0, 300, 39)) + [300]
    plens = [int(v) for v in rng.integers(0, 400, 40)]
    _check_prefix(Shared(plens, first, lens, [n] * 300, 1, 64, 16, dtype, seed=3), 4)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prefix_missing_pages(dtype):
    sh = Shared([200, 40], [0, 2, 4], [30, 0, 10, 0], [2] * 4, 2, 128, 16, dtype)
    missing = [(4, 3), (4, 4), (4, 12), (0, 0), (5, 0), (5, 1), (5, 2), (2, 0), (3, 0)]
    for i, (x, pi) in enumerate(missing):
        sh.pb.table[x, pi] = [-1, sh.pb.K.shape[0], 2 ** 31 - 1, -2 ** 31][i % 4]
    sh.bind()
    got = _check_prefix(sh, 8, missing=missing)
    assert (got[6:].float() == 0).all(), "tokens that see nothing get zeros"


def test_prefix_equals_tree_attention_over_both_parts():
    """The same keys and values in one table: the same values but for their rounding."""
    sh = Shared([512], [0, 3], [40, 3, 100], [2] * 3, 2, 128, 16)
    q = torch.randn((6, 8, 128), device="cuda").bfloat16()
    got = _run_prefix(sh, q, None)
    pb = sh.pb
    table = np.concatenate([np.repeat(pb.table[3:4, :32], 3, 0), pb.table[:3]], 1)
    cache = Q.kv_cache(pb.K, pb.V, _dev(table), _dev(np.array([552, 515, 612], np.int32)))
    O = torch.empty_like(q)
    ws = torch.empty(Q.qmm_tree_attention_workspace_bytes(cache, 8, 2), dtype=torch.uint8,
                     device="cuda")
    Q.qmm_tree_attention(cache, q, O, 2, workspace=ws)
    A = _prefix64(sh, q.cpu(), np.array([-1, 0] * 3), 1 / math.sqrt(128))[1]
    # each is within its limit of the formula's value: two roundings of the output and of
    # each weight, and FP32 work far below them
    off = (got.cpu().double() - O.cpu().double()).abs()
    assert (off <= 2 * BF16_HALF * O.cpu().double().abs() + 2.5 * BF16_HALF * A).all()


def test_prefix_of_device_values_out_of_range():
    """first, lens and cu are device data: clamped, whatever stands there; rows of no
    sequence are left alone and no answer is other than finite."""
    sh = Shared([100, 50], [0, 2, 4], [30, 7, 3, 0], [3] * 4, 2, 64, 16)
    q = torch.randn((12, 8, 64), device="cuda").bfloat16()
    nb = Q.qmm_prefix_attention_workspace_bytes(sh.cache, 8, 12, 3)
    for first in ([-5, 2, 99], [4, 2, 0], [2 ** 31 - 1, -2 ** 31, 3], [1, 1, 1]):
        for plens in ([100, 50], [-3, 2 ** 31 - 1]):
            for cu in (None, [0, 99, 3, 12, 12], [-5, 4, 8, 2 ** 31 - 1, 0], [12, 8, 4, 0, 0]):
                sh.d_first.copy_(_dev(np.asarray(first, np.int64).astype(np.int32)))
                sh.d_plens.copy_(_dev(np.asarray(plens, np.int64).astype(np.int32)))
                sh.pb.K.nan_to_num_(0.0), sh.pb.V.nan_to_num_(0.0)
                O = torch.full_like(q, 7.0)
                ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
                Q.qmm_prefix_attention(sh.cache, sh.prefix, q, O, 3, workspace=ws,
                                       cu=None if cu is None else _dev(
                                           np.asarray(cu, np.int64).astype(np.int32)))
                torch.cuda.synchronize()
                assert torch.isfinite(O.float()).all()


def test_prefix_workspace_too_small_and_other_rows():
    sh = Shared([100], [0, 2], [30, 7], [3, 2], 2, 64, 16)
    q = torch.randn((9, 8, 64), device="cuda").bfloat16()
    O = torch.full_like(q, 7.0)
    nb = Q.qmm_prefix_attention_workspace_bytes(sh.cache, 8, 9, 3)
    for ws in (None, torch.empty(nb - 16, dtype=torch.uint8, device="cuda")):
        with pytest.raises(Q.QmmError) as e:
            Q.qmm_prefix_attention(sh.cache, sh.prefix, q, O, 3, cu=_dev(sh.cu), workspace=ws)
        assert e.value.code == Q.QMM_EWORKSPACE
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    Q.qmm_prefix_attention(sh.cache, sh.prefix, q, O, 3, cu=_dev(sh.cu), workspace=ws)
    assert (O[5:] == 7.0).all() and not (O[:5] == 7.0).all(-1).any()


def test_prefix_strided_q_gets_the_same_bits():
    sh = Shared([150], [0, 2], [30, 7], [3, 2], 2, 128, 16)
    wide = torch.randn((5, 20, 128), device="cuda").bfloat16()
    a = _run_prefix(sh, wide[:, 4:12], None)
    assert _same(a, _run_prefix(sh, wide[:, 4:12].contiguous(), None))


# ---- weights by slot -----------------------------------------------------------------

def _scored64(pb, q, scale, missing=()):
    """Of a chain, in 64 bits: O, sum p |v|, the largest scale sum |q k| of a row; and by
    (sequence, head, slot) the sum of the weights and of how far each may be off."""
    N, Hq, D = q.shape
    qg = Hq // pb.Hkv
    O, A, S = (torch.zeros(s, dtype=torch.float64) for s in ((N, Hq, D), (N, Hq, D), (N, Hq)))
    W, E = [], []
    for b in range(pb.B):
        n, ln = pb.n[b], pb.lens[b]
        K, V = pb.values[0][b], pb.values[1][b]
        w, e = torch.zeros((pb.Hkv, ln + n), dtype=torch.float64), \
            torch.zeros((pb.Hkv, ln + n), dtype=torch.float64)
        there = torch.ones(ln + n, dtype=torch.bool)
        for bb, pi in missing:
            if bb == b:
                there[pi * pb.page:(pi + 1) * pb.page] = False
        for i in range(n):
            see = there.clone()
            see[ln + i + 1:] = False
            if not see.any():
                continue
            r = pb.cu[b] + i
            x = q[r].double().view(pb.Hkv, qg, D)
            s = torch.einsum("hgd,lhd->hgl", x, K[see]) * scale
            p = torch.softmax(s, -1)
            O[r] = torch.einsum("hgl,lhd->hgd", p, V[see]).reshape(Hq, D)
            A[r] = torch.einsum("hgl,lhd->hgd", p, V[see].abs()).reshape(Hq, D)
            mag = torch.einsum("hgd,lhd->hgl", x.abs(), K[see].abs()).amax(-1) * scale
            S[r] = mag.reshape(Hq)
            # a weight 2^(score - lse): FP32 scores of D products, (D + 2) 2^-24 of
            # sum |q k|, in it and in the sum; lse and the difference rounded, 2^-24 of
            # their sizes (log2 units); sums over the positions as for O; exp2 and log2
            # to 4 ulp
            lse = torch.logsumexp(s, -1) / math.log(2)
            size = 2 * lse.abs()[..., None] + s.abs() / math.log(2)
            rel = 2 * (D + 2) * F32_HALF * mag[..., None] + F32_HALF * (size + 1024 + 8)
            if pb.fp8 and pb.T * qg > 8:
                # q held to 2^-17 of its largest value where it is below 2^-9 of it, in
                # both as well
                big = x.abs().amax(-1, keepdim=True)
                small = (x.abs() < big * 2.0 ** -9).double() * big * 2.0 ** -17
                rel = rel + 2 * scale * torch.einsum("hgd,lhd->hgl", small,
                                                     K[see].abs()).amax(-1, keepdim=True)
            w[:, see] += p.sum(1)
            e[:, see] += (p * rel).sum(1) + n * qg * F32_HALF * p.sum(1) + 2.0 ** -120
        W.append(w)
        E.append(e)
    return O, A, S, W, E


def _run_scored(pb, q, mass, decay, scale=0.0, ws=None, stream=None, O=None):
    N, Hq, D = q.shape
    O = torch.full((N, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda") if O is None else O
    if ws is None:
        nb = Q.qmm_scored_attention_workspace_bytes(pb.cache, Hq, pb.T)
        ws = torch.full((nb // 4,), float("nan"), device="cuda")
    Q.qmm_scored_attention(pb.cache, q, O, pb.T, mass, decay=decay, cu=pb.cu_arg(), scale=scale,
                           workspace=ws, stream=stream)
    return O


def _check_scored(pb, Hq, decay=1.0, scale=0.0, seed=1, q_scale=2.0, missing=()):
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(q_scale * rng.standard_normal((pb.N, Hq, pb.D))).bfloat16()
    S_ = pb.width * pb.page
    old = torch.from_numpy(rng.exponential(0.3, (pb.B, pb.Hkv, S_ + 8))).float()
    for b in range(pb.B):   # the new tokens' slots, and with decay 0 all, hold anything
        old[b, :, 0 if decay == 0 else pb.lens[b]:pb.lens[b] + pb.n[b]] = float("nan")
    mass = [old.cuda() for _ in range(2)]
    got = [_run_scored(pb, q.cuda(), m, decay, scale) for m in mass]
    torch.cuda.synchronize()
    assert _same(*got) and _same(*mass), "not deterministic"
    O, A, S, W, E = _scored64(pb, q, scale or 1 / math.sqrt(pb.D), missing)
    _within(got[0].cpu(), O, _o_limit(pb.fp8, O, A, S, pb.D))
    m = mass[0].cpu()
    for b in range(pb.B):
        end, ln = pb.lens[b] + pb.n[b], pb.lens[b]
        assert _same(m[b, :, end:].contiguous(), old[b, :, end:].contiguous()), "slots behind the last"
        base = torch.zeros((pb.Hkv, end), dtype=torch.float64)
        if decay:
            base[:, :ln] = float(np.float32(decay)) * old[b, :, :ln].double()
        want = base + W[b]
        _within(m[b, :, :end], want, E[b] + 2 * F32_HALF * want)
    return got[0], mass[0]


SCORED = [
    # lens, n, Hq, Hkv, D, page, dtype, layout, decay
    ([0], [1], 1, 1, 64, 8, "bf16", "hnd", 1.0),
    ([0], [1], 4, 1, 128, 16, "e4m3", "hnd", 0.0),
    ([1000], [1], 32, 8, 128, 16, "bf16", "hnd", 0.98),
    ([1000], [1], 32, 8, 128, 16, "e4m3", "nhd", 0.98),
    ([63, 64, 65, 0, 127, 128, 129], [1] * 7, 8, 2, 128, 64, "bf16", "nhd", 1.0),
    ([63, 64, 65, 0, 127, 128, 129], [1] * 7, 16, 2, 64, 64, "e4m3", "nhd", 1.0),
    ([62, 63, 64, 0, 126, 1], [2] * 6, 4, 2, 64, 32, "bf16", "hnd", 0.5),
    ([5, 700, 0, 61], [1, 2, 0, 2], 6, 2, 128, 8, "bf16", "hnd", 0.5),
    ([5, 333, 0, 61], [7, 3, 0, 9], 6, 2, 64, 8, "e4m3", "nhd", 1.0),
    ([5, 333, 0, 61], [7, 3, 0, 9], 10, 2, 128, 8, "bf16", "nhd", 0.0),
    ([300, 3], [1, 1], 64, 2, 128, 16, "bf16", "hnd", 1.0),
    ([300, 3], [1, 1], 64, 1, 64, 16, "e4m3", "hnd", 1.0),
    ([100, 30], [64, 64], 8, 2, 128, 128, "bf16", "hnd", 0.25),
    ([100, 30], [33, 61], 21, 3, 128, 32, "e4m3", "nhd", 1.0),
    ([77, 400], [256, 200], 8, 2, 64, 64, "bf16", "nhd", 1.0),
    ([77, 400], [256, 200], 2, 2, 128, 64, "e4m3", "nhd", 0.0),
    ([20000, 3, 1500], [1, 1, 1], 8, 2, 128, 64, "bf16", "hnd", 1.0),
    ([9000, 3, 1500], [20, 1, 4], 8, 2, 64, 16, "e4m3", "nhd", 1.0),
]


@pytest.mark.parametrize("lens,n,Hq,Hkv,D,page,dtype,layout,decay", SCORED,
                         ids=["%d" % i for i in range(len(SCORED))])
def test_scored(lens, n, Hq, Hkv, D, page, dtype, layout, decay):
    _check_scored(Problem(lens, n, Hkv, D, page, dtype, layout), Hq, decay)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("e4m3", 128), ("bf16", 64), ("e4m3", 64)])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 32, 33, 64, 65, 127, 128, 129, 255, 256])
def test_scored_row_borders(rows, dtype, D):
    """One query head per KV head: as many rows as tokens."""
    _check_scored(Problem([150, 0, 64], [rows, 1, rows - 1], 2, D, 32, dtype, seed=rows), 2)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3])
def test_scored_many_sequences(n, dtype):
    rng = np.random.default_rng(5)
    lens = [int(v) for v in rng.integers(0, 90, 333)]
    _check_scored(Problem(lens, [n] * 333, 1, 64, 16, dtype, seed=3), 4)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 24])
def test_scored_missing_pages(n, dtype):
    """Positions without pages get nothing; a token that sees none gives nothing."""
    pb = Problem([200, 40, 10, 0], [n] * 4, 2, 128, 16, dtype)
    missing = [(0, 3), (0, 4), (1, 0), (2, 0), (3, 0)] + [(b, pi) for b in (2, 3) for pi in range(4)]
    for i, (b, pi) in enumerate(missing):
        pb.table[b, pi] = [-1, pb.K.shape[0], 2 ** 31 - 1, -2 ** 31][i % 4]
    pb.bind()
    _check_scored(pb, 8, 0.5, missing=missing)


def test_scored_scale_extremes():
    pb = Problem([300, 20], [1, 1], 2, 128, 32)
    _check_scored(pb, 8, scale=1e-3)
    _check_scored(pb, 8, q_scale=60.0)       # one weight takes nearly all
    pb = Problem([300, 20], [40, 40], 2, 128, 32)
    _check_scored(pb, 8, scale=1e-3)
    _check_scored(pb, 8, q_scale=60.0)
    for n in (1, 12):
        pb = Problem([300, 20], [n, n], 2, 128, 32, "e4m3", k_scale=0.3, v_scale=30.0)
        _check_scored(pb, 8, q_scale=1e-4)


@pytest.mark.parametrize("n", [1, 40])
def test_scored_output_is_tree_attentions(n):
    pb = Problem([300, 20], [n, n], 2, 128, 32)
    q = torch.randn((2 * n, 8, 128), device="cuda").bfloat16()
    mass = torch.zeros((2, 2, pb.width * 32), device="cuda")
    O = torch.empty_like(q)
    ws = torch.empty(Q.qmm_tree_attention_workspace_bytes(pb.cache, 8, n), dtype=torch.uint8,
                     device="cuda")
    Q.qmm_tree_attention(pb.cache, q, O, n, workspace=ws)
    assert _same(_run_scored(pb, q, mass, 1.0), O)
    # all of the softmax's weight arrives: 4 heads' rows, each weight to 2 (D + 2) 2^-24 of
    # sum |q k| < 60 and the sums' roundings
    total = mass.double().sum(-1)
    assert ((total - 4 * n).abs() <= 4 * n * 2.0 ** -10).all()


@pytest.mark.parametrize("n", [1, 24])
def test_scored_not_numbers_and_workspace(n):
    """NaN in q reaches the weights of its sequence's head alone; too small a workspace
    is refused."""
    pb = Problem([130, 5], [n, n], 2, 128, 16)
    q = torch.randn((pb.N, 8, 128), device="cuda").bfloat16()
    mass = torch.zeros((2, 2, pb.width * 16), device="cuda")
    clean = mass.clone()
    _run_scored(pb, q, clean, 1.0)
    bad = q.clone()
    bad[0, 1, 5] = float("nan")              # sequence 0, KV head 0
    _run_scored(pb, bad, mass, 1.0)
    assert _same(mass[1], clean[1]) and _same(mass[0, 1], clean[0, 1])
    assert torch.isnan(mass[0, 0, :131]).all() and _same(mass[0, 0, 130 + n:], clean[0, 0, 130 + n:])
    nb = Q.qmm_scored_attention_workspace_bytes(pb.cache, 8, n)
    for ws in (None, torch.empty(nb - 16, dtype=torch.uint8, device="cuda")):
        with pytest.raises(Q.QmmError) as e:
            Q.qmm_scored_attention(pb.cache, q, torch.empty_like(q), n, mass, workspace=ws)
        assert e.value.code == Q.QMM_EWORKSPACE


# ---- eviction --------------------------------------------------------------------------

def _kept(mass, ln, keep, sinks, recent):
    """The slot whose rows stand in each of the first min(ln, keep) slots."""
    if ln <= keep:
        return np.arange(ln)
    middle = np.arange(sinks, ln - recent)
    w = np.where(np.isnan(mass[middle]), -np.inf, mass[middle].astype(np.float64))
    nan = np.isnan(mass[middle])
    order = sorted(range(len(middle)), key=lambda i: (nan[i], -w[i], middle[i]))
    best = {int(middle[i]) for i in order[:keep - sinks - recent]}
    line = keep - recent
    late = sorted(i for i in best if i >= line)
    out = [i if i < sinks or i in best else late.pop(0) for i in range(line)]
    assert not late
    return np.array(out + list(range(ln - recent, ln)))


def _check_evict(lens, keep, sinks, recent, Hkv=2, D=64, page=16, dtype="bf16", layout="hnd",
                 layers=1, kind="spread", in_place=False, missing=(), seed=0, stride=0):
    rng = np.random.default_rng(seed)
    B = len(lens)
    width = -(-max(max(lens), 1) // page) + 1
    pages = sum(-(-x // page) for x in lens) + 3
    ids = iter(rng.permutation(pages))
    table = np.full((B, width), -1, np.int32)
    for b, ln in enumerate(lens):
        m = -(-ln // page)
        table[b, :m] = [next(ids) for _ in range(m)]
    for b, pi in missing:
        table[b, pi] = [-1, pages, 2 ** 31 - 1][pi % 3]
    fp8 = dtype == "e4m3"
    shape = (layers, pages, Hkv, page, D) if layout == "hnd" else (layers, pages, page, Hkv, D)
    bits = torch.uint8 if fp8 else torch.int16
    pools = [torch.from_numpy(rng.integers(0, 256, shape + ((1,) if fp8 else (2,)),
                                           dtype=np.uint8)).view(bits).squeeze(-1) for _ in "kv"]
    dev = [p.cuda().view(torch.float8_e4m3fn if fp8 else torch.bfloat16) for p in pools]
    views = [(d if layout == "hnd" else d.transpose(2, 3)) for d in dev]
    S = width * page + stride
    mass = rng.exponential(1.0, (layers, B, Hkv, S)).astype(np.float32)
    if kind == "ties":
        mass = rng.integers(0, 4, mass.shape).astype(np.float32)
    elif kind == "equal":
        mass[:] = 0.5
    elif kind == "odd":
        odd = np.array([0.0, -0.0, np.nan, np.inf, -np.inf, -1.5, 1e-45, -1e-45, 3e38], np.float32)
        mass = odd[rng.integers(0, len(odd), mass.shape)]
    elif kind == "near":   # neighbours in FP32: all bits decide
        mass = (np.float32(1.0).view(np.int32) + rng.integers(0, 300, mass.shape)).astype(
            np.int32).view(np.float32)
    elif kind == "rising":
        mass = np.broadcast_to(np.arange(S, dtype=np.float32), mass.shape).copy()
    elif kind == "falling":
        mass = np.broadcast_to(-np.arange(S, dtype=np.float32), mass.shape).copy()
    d_lens, d_table = _dev(np.asarray(lens, np.int32)), _dev(table)
    caches = Q.kv_caches([Q.kv_cache(views[0][i], views[1][i], d_table, d_lens,
                                     *((0.5, 2.0) if fp8 else (1.0, 1.0))) for i in range(layers)])
    d_mass = torch.from_numpy(mass).cuda()
    out = d_mass if in_place else torch.full_like(d_mass, 9.0)
    kept = torch.full((layers, B, Hkv, keep), -7, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    Q.qmm_kv_evict(caches, d_mass, keep, kept, new, sinks=sinks, recent=recent,
                   mass_out=None if in_place else out)
    torch.cuda.synchronize()
    assert new.tolist() == [min(x, keep) for x in lens] and d_lens.tolist() == list(lens)
    want = [p.clone() for p in pools]
    w_out = mass.copy() if in_place else np.full_like(mass, 9.0)
    w_kept = np.full(kept.shape, -1, np.int64)
    for la in range(layers):
        for b, ln in enumerate(lens):
            for h in range(Hkv):
                k = _kept(mass[la, b, h], ln, keep, sinks, recent)
                w_kept[la, b, h, :len(k)] = k
                w_out[la, b, h, :len(k)] = mass[la, b, h, k]
                for j, s in enumerate(k):
                    ps, pd = table[b, s // page], table[b, j // page]
                    if s == j or not (0 <= ps < pages and 0 <= pd < pages):
                        continue
                    for x, y in zip(pools, want):
                        if layout == "hnd":
                            y[la, pd, h, j % page] = x[la, ps, h, s % page]
                        else:
                            y[la, pd, j % page, h] = x[la, ps, s % page, h]
    assert torch.equal(kept.cpu().long(), torch.from_numpy(w_kept))
    assert np.array_equal(out.cpu().numpy().view(np.int32), w_out.view(np.int32))
    if not in_place:
        assert np.array_equal(d_mass.cpu().numpy().view(np.int32), mass.view(np.int32))
    for d, y in zip(dev, want):
        assert torch.equal(d.view(bits).cpu(), y)


EVICT = [
    # lens, keep, sinks, recent
    ([0, 1, 2, 3], 1, 0, 0), ([0, 1, 2, 3], 1, 1, 0), ([0, 1, 2, 3], 1, 0, 1),
    ([31, 32, 33, 34], 32, 0, 0), ([31, 32, 33, 34], 32, 4, 28), ([31, 32, 33, 34], 32, 32, 0),
    ([31, 32, 33, 34], 32, 0, 32), ([200, 90, 40, 33], 32, 3, 8), ([200, 90, 40, 33], 32, 0, 20),
    ([1500, 513, 1025, 700], 512, 4, 128), ([1500, 513, 1025, 700], 512, 4, 500),
    ([600, 513, 514, 620], 512, 0, 511), ([2000, 1537], 1536, 4, 1000), ([5000, 3000], 700, 1, 0),
]


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("lens,keep,sinks,recent", EVICT, ids=["%d" % i for i in range(len(EVICT))])
def test_evict(lens, keep, sinks, recent, kind):
    _check_evict(lens, keep, sinks, recent, kind=kind, in_place=kind == "ties", seed=keep)


@pytest.mark.parametrize("kind", ["equal", "near", "rising", "falling"])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_orders(kind, in_place):
    _check_evict([1300, 900], 800, 4, 60, kind=kind, in_place=in_place)
    _check_evict([1300, 900], 300, 0, 299, kind=kind, in_place=in_place)


@pytest.mark.parametrize("D,dtype,layout,page,layers", [
    (128, "bf16", "hnd", 16, 3), (128, "bf16", "nhd", 8, 2), (64, "e4m3", "nhd", 64, 2),
    (64, "e4m3", "hnd", 8, 1), (128, "e4m3", "nhd", 128, 2), (64, "bf16", "nhd", 32, 70)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_layouts(D, dtype, layout, page, layers, in_place):
    _check_evict([90, 300, 20], 64, 2, 16, 3, D, page, dtype, layout, layers, in_place=in_place,
                 stride=20 if layers == 2 else 0)


def test_evict_missing_pages():
    _check_evict([300, 200], 100, 3, 30, missing=[(0, 1), (0, 4), (0, 9), (0, 18), (1, 3), (1, 12)])


@pytest.mark.parametrize("lens,keep,sinks,recent,Hkv,kind,in_place", [
    ([140000, 70001, 131073], 40000, 4, 9000, 1, "near", True),   # beyond eight blocks' memory
    ([131072, 131071, 100000], 70000, 0, 1, 1, "ties", False),
    ([16384], 5000, 3, 100, 2, "ties", True), ([16385], 16000, 0, 0, 2, "odd", False),
    ([40000, 33000, 16000, 300], 8000, 4, 500, 1, "equal", True),
    ([40000, 33000, 16000, 300], 20000, 4, 0, 1, "odd", True),
    ([9000], 33, 1, 32, 1, "spread", False), ([9000], 8999, 0, 8999, 1, "spread", True),
    ([9000], 8990, 17, 70, 3, "rising", True), ([9000], 4500, 17, 70, 3, "falling", False),
    ([4097], 64, 0, 0, 1, "near", True), ([30000], 10, 0, 10, 1, "ties", False),
])
def test_evict_long_rows(lens, keep, sinks, recent, Hkv, kind, in_place):
    """Columns that several blocks share, and longer ones that go through memory."""
    _check_evict(lens, keep, sinks, recent, Hkv, 64, 64, "e4m3", kind=kind, in_place=in_place)


@pytest.mark.parametrize("dtype,D,layout", [("bf16", 128, "nhd"), ("bf16", 64, "hnd"), ("e4m3", 128, "hnd")])
def test_evict_rows_in_pieces_by_several_blocks(dtype, D, layout):
    """Few columns: a row's pieces and the parts of a batch go to different blocks, and rows
    that move by less than a batch."""
    _check_evict([9000], 8990, 17, 70, 2, D, 16, dtype, layout, kind="spread", in_place=True)
    _check_evict([5000, 4000], 3900, 0, 3000, 1, D, 32, dtype, layout, kind="ties")


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_short_columns_of_a_long_table(in_place):
    """Columns in fewer slots than their cluster has blocks, beside one that needs them all."""
    _check_evict([40000, 3, 0, 33, 1100], 30, 2, 11, 1, kind="ties", in_place=in_place)
    _check_evict([1, 65, 140000, 31, 32], 31, 31, 0, 1, page=64, in_place=in_place)
    _check_evict([32, 64, 20000, 96], 1, 0, 0, 2, page=32, kind="odd", in_place=in_place)


def test_evict_long_tables_of_many_columns():
    """Tables far longer than what stands in them: a block a column, the others leave."""
    _check_evict([600, 20000, 33, 16385] * 5, 500, 4, 60, 8, 64, 64, "e4m3", kind="ties",
                 in_place=True)


def test_evict_clamps_lens_to_the_table():
    c = Problem([60, 3], [0, 0], 1, 64, 16, width=4)
    c.lens = [2 ** 31 - 1, -5]
    c.bind()
    mass = torch.rand((2, 1, 64), device="cuda")
    kept = torch.empty((1, 2, 1, 50), dtype=torch.int32, device="cuda")
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    Q.qmm_kv_evict(Q.kv_caches([c.cache]), mass.clone(), 50, kept, new, sinks=1, recent=9)
    assert new.tolist() == [50, 0] and (kept[0, 1] == -1).all()
    assert kept[0, 0, 0].tolist() == _kept(mass[0, 0].cpu().numpy(), 64, 50, 1, 9).tolist()


# ---- positions of several axes ----------------------------------------------------------

def _axes_case(lens, n, Hq, Hkv, D, page, dtype, layout, rot, inter, norm, axis, A, seed=9):
    pb = Problem(lens, n, Hkv, D, page, dtype, layout)
    rng = np.random.default_rng(seed)
    N = pb.N
    x = torch.from_numpy(rng.standard_normal((N, Hq + 2 * Hkv, D)) *
                         np.exp(rng.standard_normal((N, 1, 1)))).bfloat16()
    rows = 200
    cs = _cos_sin(rows, rot)
    w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).bfloat16() if norm else None for _ in "qk"]
    pos = rng.integers(0, rows, (A, N))
    return pb, x, cs, w, pos, Q.rope(cs.cuda(), inter, *(None if t is None else t.cuda() for t in w),
                                     1e-5), Q.rope_axes(axis, A)


def _turned_axes(x, w, cs, pos, axis, inter, eps):
    """Norm and rotation in 64 bits, and the sum of the magnitudes that go in."""
    x = x.double().clone()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    mag, half = x.abs(), cs.shape[1] // 2
    for j, a in enumerate(axis):
        row = cs[torch.from_numpy(pos[a])].double()
        c, s = row[:, j, None], row[:, half + j, None]
        u, v = (2 * j, 2 * j + 1) if inter else (j, j + half)
        p, q = x[..., u].clone(), x[..., v].clone()
        x[..., u], x[..., v] = p * c - q * s, q * c + p * s
        mag[..., u], mag[..., v] = p.abs() * c.abs() + q.abs() * s.abs(), \
            q.abs() * c.abs() + p.abs() * s.abs()
    return x, mag


AXES = [
    # lens, n, Hq, Hkv, D, page, dtype, layout, rot, interleaved, norm, axis of each pair, axes
    ([0], [1], 1, 1, 64, 8, "bf16", "hnd", 64, False, False, [0] * 8 + [1] * 12 + [2] * 12, 3),
    ([1000], [1], 32, 8, 128, 16, "bf16", "hnd", 128, False, True, [0] * 16 + [1] * 24 + [2] * 24, 3),
    ([15, 0, 100], [5, 40, 1], 6, 2, 128, 16, "e4m3", "nhd", 128, False, True,
     [j % 3 for j in range(64)], 3),
    ([15, 0, 100], [5, 0, 41], 3, 1, 64, 32, "e4m3", "hnd", 16, False, False,
     [7, 0, 3, 1, 5, 2, 6, 4], 8),
    ([15, 0, 100], [5, 0, 41], 5, 5, 64, 8, "bf16", "hnd", 32, True, False,
     [j // 5 % 2 for j in range(16)], 2),
    ([7] * 40, [3] * 40, 0, 4, 128, 64, "bf16", "nhd", 64, True, True, [1] * 32, 5),
    ([1, 2], [700, 300], 24, 8, 64, 128, "bf16", "nhd", 48, False, True,
     [j % 4 for j in range(24)], 4),
]


@pytest.mark.parametrize("lens,n,Hq,Hkv,D,page,dtype,layout,rot,inter,norm,axis,A", AXES,
                         ids=["%d" % i for i in range(len(AXES))])
def test_axes(lens, n, Hq, Hkv, D, page, dtype, layout, rot, inter, norm, axis, A):
    pb, x, cs, w, pos, rope, axes = _axes_case(lens, n, Hq, Hkv, D, page, dtype, layout, rot, inter,
                                               norm, axis, A)
    N, xd = pb.N, x.cuda()
    old = [t.view(torch.int8 if pb.fp8 else torch.int16).clone() for t in (pb.K, pb.V)]
    out = torch.full((N, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda") if Hq else None
    Q.qmm_kv_append_axes(pb.cache, xd[:, :Hq] if Hq else None, xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:],
                         _dev(pos.astype(np.int32)), axes, rope, q_out=out, cu=pb.cu_arg())
    torch.cuda.synchronize()
    if Hq:
        assert _near_bf16(out, *_turned_axes(x[:, :Hq], w[0], cs, pos, axis, inter, 1e-5))
    wk, mk = _turned_axes(x[:, Hq:Hq + Hkv], w[1], cs, pos, axis, inter, 1e-5)
    wv = x[:, Hq + Hkv:].double()
    seq = np.repeat(np.arange(pb.B), n)
    slot = np.asarray(lens)[seq] + np.arange(N) - pb.cu[seq]
    at = (torch.from_numpy(pb.table[seq, slot // page]).long().cuda(), slice(None),
          torch.from_numpy(slot % page).cuda())
    for i, (pool, want, mag) in enumerate(((pb.K, wk, mk), (pb.V, wv, wv.abs()))):
        b = pool.view(torch.int8 if pb.fp8 else torch.int16)
        got = b[at].view(pool.dtype).float()
        if pb.fp8:
            sc = float(np.float32(pb.scales[i]))
            assert _near_e4m3(got, want / sc, mag / sc)
        elif i == 1:
            assert torch.equal(got.cpu().double(), want)
        else:
            assert _near_bf16(got, want, mag)
        keep = b.clone()
        keep[at] = old[i][at]
        assert torch.equal(keep, old[i]), "other rows of the pool"


@pytest.mark.parametrize("D,inter,dtype", [(128, False, "bf16"), (64, True, "e4m3"),
                                           (128, True, "bf16"), (64, False, "bf16")])
def test_axes_that_agree_are_plain_positions(D, inter, dtype):
    """One axis, or several with the same positions: qmm_kv_append's bits."""
    for axis, A in (([0] * (D // 2), 1), ([j % 3 for j in range(D // 2)], 3)):
        got = []
        for plain in (False, True):
            pb, x, cs, w, pos, rope, axes = _axes_case([5, 30, 0], [7, 2, 9], 8, 2, D, 16, dtype,
                                                       "hnd", D, inter, True, axis, A)
            pos[:] = pos[0]
            xd, d_pos = x.cuda(), _dev(pos.astype(np.int32))
            out = torch.empty((pb.N, 8, D), dtype=torch.bfloat16, device="cuda")
            args = (pb.cache, xd[:, :8], xd[:, 8:10], xd[:, 10:])
            if plain:
                Q.qmm_kv_append(*args, out, rope=rope, positions=d_pos[0].contiguous(),
                                cu=pb.cu_arg())
            else:
                Q.qmm_kv_append_axes(*args, d_pos, axes, rope, q_out=out, cu=pb.cu_arg())
            got.append([out] + [t.view(torch.int8 if pb.fp8 else torch.int16) for t in (pb.K, pb.V)])
        assert all(torch.equal(a.view(b.dtype), b) for a, b in zip(*got))


def test_axes_any_position_off_the_table_leaves_the_token():
    pb, x, cs, w, pos, rope, axes = _axes_case([10, 5], [4, 4], 4, 2, 128, 16, "bf16", "hnd", 32,
                                               False, True, [0] * 8 + [2] * 8, 4)
    pos[:, [0, 4]] = 7
    pos[0, 1], pos[2, 2], pos[3, 3], pos[1, 5], pos[2, 6], pos[0, 7] = -1, 200, 2 ** 31 - 1, \
        -2 ** 31, -9, 200
    xd, old = x.cuda(), pb.K.view(torch.int16).clone()
    out = torch.full((8, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    Q.qmm_kv_append_axes(pb.cache, xd[:, :4], xd[:, 4:6], xd[:, 6:], _dev(pos.astype(np.int32)),
                         axes, rope, q_out=out)
    for t in range(8):
        b, i = divmod(t, 4)
        s = pb.lens[b] + i
        at = (int(pb.table[b, s // 16]), slice(None), s % 16)
        left = t not in (0, 4)
        assert bool((out[t] == 5.0).all()) == left
        assert torch.equal(pb.K.view(torch.int16)[at], old[at]) == left
    # in place: q's own rows
    y = x.cuda()
    Q.qmm_kv_append_axes(pb.cache, y[:, :4], y[:, 4:6], y[:, 6:], _dev(pos.astype(np.int32)), axes,
                         rope, q_out=y[:, :4])
    assert torch.equal(y[[0, 4], :4], out[[0, 4]])
    assert torch.equal(y[[1, 2, 3, 5, 6, 7]], xd[[1, 2, 3, 5, 6, 7]])


# ---- together -----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,graph", [("bf16", False), ("bf16", True), ("e4m3", False)])
def test_steps_with_eviction(dtype, graph):
    """A prompt, its last tokens as the first window, then steps of append - scored
    attention and an eviction every third one, in two layers, against a history of the
    rows that stay, kept by head in 64 bits.  Positions go on counting."""
    rng = np.random.default_rng(12)
    B, Hq, Hkv, D, page, layers, keep, sinks, recent, window = 2, 8, 2, 64, 16, 2, 40, 2, 10, 5
    prompt = [61, 33]
    cap, steps = 96, 9
    width = cap // page
    fp8 = dtype == "e4m3"
    scales = (0.02, 0.015) if fp8 else (1.0, 1.0)
    table = _dev(rng.permutation(B * width).reshape(B, width).astype(np.int32))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.zeros_like(lens)
    caches = []
    for _ in range(layers):
        pools = [torch.full((B * width, Hkv, page, D), float("nan"), device="cuda").to(
            torch.float8_e4m3fn if fp8 else torch.bfloat16) for _ in "kv"]
        caches.append(Q.kv_cache(*pools, table, lens, *scales))
    group = Q.kv_caches(caches)
    axis = [j % 2 for j in range(D // 2)]
    cs = _cos_sin(400, D)
    rope, axes = Q.rope(cs.cuda()), Q.rope_axes(axis)
    mass = torch.full((layers, B, Hkv, cap), float("nan"), device="cuda")
    kept = torch.zeros((layers, B, Hkv, keep), dtype=torch.int32, device="cuda")

    def pool_rows(la, b, m):
        """The rows that stand in the cache, by head: [2][Hkv, m, D] in 64 bits."""
        out = []
        for pool, sc in zip(caches[la].tensors[:2], scales):
            s = torch.arange(m, device="cuda")
            r = pool.view(torch.uint8 if fp8 else torch.int16)[table[b].long()[s // page], :, s % page]
            out.append(r.view(pool.dtype).double().cpu().transpose(0, 1) * sc)
        return out

    cu = np.concatenate([[0], np.cumsum(prompt)]).astype(np.int32)
    qs = []
    for la in range(layers):
        x = torch.from_numpy(rng.standard_normal((cu[-1], Hq + 2 * Hkv, D))).bfloat16()
        pos = np.concatenate([np.arange(m) for m in prompt])
        xd = x.cuda()
        q_out = torch.empty_like(xd[:, :Hq])
        Q.qmm_kv_append_axes(caches[la], xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:],
                             _dev(np.stack([pos, pos // 3]).astype(np.int32)), axes, rope,
                             q_out=q_out, cu=_dev(cu))
        qs.append(q_out)
    # the window: the last tokens' keys are in the cache, behind prompt - window others
    lens.copy_(_dev(np.asarray(prompt, np.int32) - window))
    ws = torch.empty(max(Q.qmm_scored_attention_workspace_bytes(caches[0], Hq, t)
                         for t in (1, window)), dtype=torch.uint8, device="cuda")
    want_mass = np.zeros((layers, B, Hkv, cap))
    rows = [[pool_rows(la, b, prompt[b]) for b in range(B)] for la in range(layers)]

    def attend64(q, la, b, ln, n):
        K, V = rows[la][b]
        out = []
        for i in range(n):
            s = torch.einsum("hgd,hld->hgl", q[i].double().view(Hkv, -1, D),
                             K[:, :ln + i + 1]) / math.sqrt(D)
            p = s.softmax(-1)
            out.append((torch.einsum("hgl,hld->hgd", p, V[:, :ln + i + 1]).reshape(Hq, D),
                        torch.einsum("hgl,hld->hgd", p, V[:, :ln + i + 1].abs()).reshape(Hq, D)))
            if i == 0:
                want_mass[la, b, :, ln:ln + n] = 0
            want_mass[la, b, :, :ln + i + 1] += p.sum(1).numpy()
        return out

    def check(O, q, la, n):
        for b in range(B):
            ln = int(lens[b])
            for i, (o, a) in enumerate(attend64(q[b], la, b, ln, n)):
                got = O[b * n + i].cpu().double()
                # q and the rows are the stored ones: the weights' rounding and FP32 work
                assert ((got - o).abs() <= BF16_HALF * o.abs() + a * (BF16_HALF + 2.0 ** -11)).all()
            m = mass[la, b, :, :ln + n].cpu().double().numpy()
            # FP32 work: 2 (D + 2) 2^-24 of sum |q k| < 30, sums of at most 1024 terms
            assert (np.abs(m - want_mass[la, b, :, :ln + n]) <=
                    2.0 ** -11 * want_mass[la, b, :, :ln + n] + 1e-30).all()

    for la in range(layers):
        q = torch.cat([qs[la][cu[b + 1] - window:cu[b + 1]] for b in range(B)]).contiguous()
        O = torch.empty_like(q)
        Q.qmm_scored_attention(caches[la], q, O, window, mass[la], decay=0.0, workspace=ws)
        check(O, q.cpu().view(B, window, Hq, D), la, window)
    lens.copy_(_dev(np.asarray(prompt, np.int32)))
    x_d = torch.zeros((layers, B, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    pos_d = torch.zeros((2, B), dtype=torch.int32, device="cuda")
    out_d = torch.zeros((layers, B, Hq, D), dtype=torch.bfloat16, device="cuda")
    q_d = torch.zeros_like(out_d)

    def step():
        for la in range(layers):
            x = x_d[la]
            Q.qmm_kv_append_axes(caches[la], x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], pos_d,
                                 axes, rope, q_out=q_d[la])
            Q.qmm_scored_attention(caches[la], q_d[la], out_d[la], 1, mass[la], workspace=ws)

    def evict():
        Q.qmm_kv_evict(group, mass, keep, kept, new, sinks=sinks, recent=recent)
        lens.copy_(new)

    graphs = None
    if graph:
        before = lens.clone()
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
        for g, f in zip(graphs, (step, evict)):
            with torch.cuda.graph(g):
                f()
        assert torch.equal(before, lens)
    for t in range(steps):
        x_d.copy_(torch.from_numpy(rng.standard_normal(x_d.shape)).bfloat16())
        pos_d.copy_(_dev(np.array([[m + t for m in prompt], [t // 2 + 50] * B], np.int32)))
        graphs[0].replay() if graph else step()
        torch.cuda.synchronize()
        for la in range(layers):
            for b in range(B):
                rows[la][b] = pool_rows(la, b, int(lens[b]) + 1)
            check(out_d[la], q_d[la].cpu().view(B, 1, Hq, D), la, 1)
        lens.add_(1)
        if t % 3 == 2:
            old, ln_old = mass.cpu().numpy(), lens.tolist()
            graphs[1].replay() if graph else evict()
            torch.cuda.synchronize()
            for la in range(layers):
                for b in range(B):
                    now = pool_rows(la, b, int(lens[b]))
                    for h in range(Hkv):
                        k = _kept(old[la, b, h], ln_old[b], keep, sinks, recent)
                        assert kept[la, b, h, :len(k)].tolist() == k.tolist()
                        want_mass[la, b, h, :len(k)] = want_mass[la, b, h, k]
                        for i in range(2):
                            assert torch.equal(now[i][h], rows[la][b][i][h][k])
                    assert int(lens[b]) == min(ln_old[b], keep)


def test_prefix_steps_with_accepted_paths():
    """Draft - append - attend behind the shared prefix - accept, against 64 bits."""
    rng = np.random.default_rng(3)
    Hq, Hkv, D, page, T, plen = 8, 2, 128, 16, 5, 90
    sh = Shared([plen], [0, 3], [20, 0, 7], [0, 0, 0], Hkv, D, page, width=12, spare=40)
    pb = sh.pb
    free = sorted(set(range(pb.K.shape[0])) - set(pb.table[pb.table >= 0].tolist()))
    for b in range(3):       # pages for what will be appended
        for j in range(12):
            if pb.table[b, j] < 0 and free:
                pb.table[b, j] = free.pop()
    sh.T = T
    sh.bind()
    new, count = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    path = torch.zeros((3, T), dtype=torch.int32, device="cuda")
    ws = torch.empty(Q.qmm_prefix_attention_workspace_bytes(sh.cache, Hq, 3 * T, T),
                     dtype=torch.uint8, device="cuda")
    for _ in range(4):
        x = torch.from_numpy(rng.standard_normal((3 * T, Hq + 2 * Hkv, D))).bfloat16()
        par = [_tree(rng, T, "tree") for _ in range(3)]
        tok, tgt = (rng.integers(0, 2, 3 * T).astype(np.int32) for _ in range(2))
        xd, d_par = x.cuda(), _dev(np.concatenate(par).astype(np.int32))
        q, O = xd[:, :Hq], torch.empty((3 * T, Hq, D), dtype=torch.bfloat16, device="cuda")
        Q.qmm_kv_append(sh.cache, None, xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:])
        Q.qmm_prefix_attention(sh.cache, sh.prefix, q, O, T, parents=d_par, workspace=ws)
        Q.qmm_tree_accept(Q.kv_caches([sh.cache]), _dev(tok), _dev(tgt), T, path, count,
                          new_lens=new, parents=d_par)
        torch.cuda.synchronize()
        sh.n, sh.cu = [T] * 3, np.arange(4) * T
        was = [[pb.values[i][b] for b in range(3)] for i in range(2)]
        for b in range(3):
            for i in range(2):
                rows = x[b * T:(b + 1) * T, Hq + i * Hkv:Hq + (i + 1) * Hkv].double()
                pb.values[i][b] = torch.cat([was[i][b], rows])
        O64, A, S = _prefix64(sh, x[:, :Hq], np.concatenate(par), 1 / math.sqrt(D))
        assert ((O.cpu().double() - O64).abs() <= _o_limit(False, O64, A, S, D)).all()
        for b in range(3):
            kept = [i for i in path[b].tolist() if i >= 0]
            for i in range(2):
                rows = pb.values[i][b][sh.lens[b]:]
                pb.values[i][b] = torch.cat([was[i][b], rows[kept]])
            sh.lens[b] += len(kept)
        sh.d_lens.copy_(new)
        assert sh.d_lens.tolist() == sh.lens


def _calls(n, seed):
    """A prefix, a scored and an evict call with fixed inputs: functions of the stream
    that run them into buffers of their own, and those buffers."""
    torch.manual_seed(seed)
    sh = Shared([300, 40], [0, 2, 3], [90, 3, 20], [n] * 3, 2, 128, 16, seed=seed)
    pb = Problem([900, 40, 333], [n] * 3, 2, 128, 16, seed=seed)
    q = torch.randn((3 * n, 8, 128), device="cuda").bfloat16()
    O, O2 = torch.zeros_like(q), torch.zeros_like(q)
    start = torch.rand((3, 2, pb.width * 16), device="cuda")
    mass = start.clone()
    kept = torch.zeros((1, 3, 2, 64), dtype=torch.int32, device="cuda")
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.empty(Q.qmm_prefix_attention_workspace_bytes(sh.cache, 8, 3 * n, n),
                     dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(Q.qmm_scored_attention_workspace_bytes(pb.cache, 8, n), dtype=torch.uint8,
                      device="cuda")
    # (its own pools: eviction moves their rows)
    ev = Problem([200, 64, 130], [0] * 3, 2, 64, 16, "e4m3", seed=seed)
    weights = torch.rand((1, 3, 2, ev.width * 16), device="cuda")
    out = torch.zeros_like(weights)
    group = Q.kv_caches([ev.cache])
    start2 = [t.view(torch.uint8).clone() for t in (ev.K, ev.V)]

    def run(stream=None):
        Q.qmm_prefix_attention(sh.cache, sh.prefix, q, O, n, workspace=ws, stream=stream)
        Q.qmm_scored_attention(pb.cache, q, O2, n, mass, decay=0.0, workspace=ws2, stream=stream)
        Q.qmm_kv_evict(group, weights, 64, kept, new, sinks=2, recent=20, mass_out=out,
                       stream=stream)

    def reset():
        for t, v in zip((ev.K, ev.V), start2):
            t.view(torch.uint8).copy_(v)
        mass.copy_(start)
        for t in (O, O2, out, kept, new):
            t.zero_()
        torch.cuda.synchronize()

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (O.view(torch.int16), O2.view(torch.int16), mass, out, kept, new,
                                    ev.K.view(torch.uint8), ev.V.view(torch.uint8))]
    run.keep = (sh, pb, ev, ws, ws2, q, weights, group)
    return run, reset, results


@pytest.mark.parametrize("n", [1, 12, 40])
def test_streams_graphs_and_threads(n):
    """Calls on streams of their own, captured and replayed side by side, from host
    threads and without programmatic launch: the eager call's bits each time."""
    import threading
    jobs = [_calls(n, s) for s in (1, 2)]
    wants = []
    for run, reset, results in jobs:
        reset()
        run()
        wants.append(results())

    def check():
        for (_, reset, results), want in zip(jobs, wants):
            assert all(torch.equal(a, b) for a, b in zip(results(), want))
            reset()

    for _, reset, _ in jobs:
        reset()
    streams = [torch.cuda.Stream() for _ in jobs]
    for (run, _, _), st in zip(jobs, streams):
        with torch.cuda.stream(st):
            run()
    check()
    graphs = []
    for run, _, _ in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    check_first = [r() for _, _, r in jobs]
    assert all(not t.any() for t in check_first[0][:2]), "a capture runs nothing"
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        check()
    errors = []

    def work(run, st):
        try:
            run(st.cuda_stream)
            st.synchronize()
        except Exception as e:                                  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(run, st)) for (run, _, _), st in zip(jobs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    check()
    Q.qmm_set_pdl(0)
    try:
        for run, _, _ in jobs:
            run()
        torch.cuda.synchronize()
    finally:
        Q.qmm_set_pdl(1)
    check()
