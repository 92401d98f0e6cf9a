"""Paged-cache calls on a GB300 at the borders of their numbers and their memory."""
import math

import numpy as np
import pytest
import torch

from split_w4a16_quantized_gb300 import qmm as Q
from test_paged_gpu import BF16_HALF, F16_HALF, F32_HALF, Problem, _attention64, _check_attention, \
    _dev, _run_attention, _tree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    yield
    torch.cuda.synchronize()
    assert Q.qmm_kernel_status(clear=True) == 0


def _set_rows(pb, pool, values):
    """One sequence's rows: values [lens + n, Hkv, D] of what its cache stores."""
    for s in range(len(values)):
        (pb.K, pb.V)[pool][int(pb.table[0, s // pb.page]), :, s % pb.page] = \
            values[s].float().to(pb.K.dtype).cuda()
    pb.values[pool][0] = values.double() * pb.scales[pool]


# ---- values of q far below the largest of their head -----------------------------

@pytest.mark.parametrize("n,D", [(1, 128), (12, 128), (12, 64), (80, 128)])
def test_small_values_of_q_beside_a_large_one(n, D):
    """E4M3 cache: q holds one value of 128, where the keys are zero, and one small
    value c elsewhere, where they are +-448: scores are all made of c.  c is held
    to 2^-17 of the row's largest value, and exactly from 2^-9 of it on."""
    pb = Problem([96], [n], 2, D, 16, "e4m3", seed=2, k_scale=2.0 ** -10, v_scale=2.0 ** -6)
    rng = np.random.default_rng(n)
    sign = np.where(np.arange(96 + n) % 2 == 0, 1.0, -1.0)
    k = torch.from_numpy(np.broadcast_to(448.0 * sign[:, None, None], (96 + n, 2, D)).copy())
    k[:, :, 0] = 0
    v = torch.from_numpy(np.broadcast_to(64.0 * sign[:, None, None], (96 + n, 2, D)).copy())
    _set_rows(pb, 0, k)
    _set_rows(pb, 1, v)
    # 8-bit significands 2^-12 to 2^-1; among them 0.0097046, whose 4 leading bits
    # alone lie between two E4M3 numbers
    c = rng.integers(128, 256, (n, 4)) * 2.0 ** (-7 - rng.integers(1, 12, (n, 4)))
    c[0, 0] = 159 * 2.0 ** -14
    q = torch.from_numpy(np.broadcast_to(c[:, :, None], (n, 4, D)).copy()).bfloat16()
    assert (q[:, :, 1].double().numpy() == c).all()
    q[:, :, 0] = 128.0
    parents = np.arange(-1, n - 1).astype(np.int32)
    # scale such that c's allowed error moves a score by 0.05
    worst = (D - 1) * 448 * 2.0 ** -10                 # |key| of a score, as stored
    scale = 0.05 / (worst * 128 * 2.0 ** -17)
    got = _run_attention(pb, q.cuda(), parents, scale).cpu().double()
    O, _, S = _attention64(pb, q, parents, scale)
    # each score off by delta at most (c's rounding, 0 from 2^-9 on, and FP32:
    # (D + 2) 2^-24 of sum |q k|): weights by a factor within exp(+-delta), and as
    # |V| = 1, sum p |v - O| = 1 - O^2 takes it to O.  Second order: delta^2.
    # Then F16 weights, sums below 2^-24 * 1024, and O's own rounding.
    small = torch.from_numpy(c) < 128 * 2.0 ** -9
    delta = (torch.where(small, 0.05, 0.0) + 2 * (D + 2) * F32_HALF * S)[..., None]
    lim = BF16_HALF * O.abs() + (1 - O * O) * delta + delta ** 2 + F16_HALF + 1024 * F32_HALF
    off = (got - O).abs()
    assert (off <= lim).all(), (off / lim).max()


@pytest.mark.parametrize("n,D", [(1, 128), (12, 128), (12, 64), (80, 128)])
def test_largest_values_of_q(n, D):
    """E4M3 cache, values of q in the last binade that BF16 has: 249 and -223 times
    2^120 against the same key, so that the score is made of their difference."""
    ks = 2.0 ** -60
    pb = Problem([96], [n], 2, D, 16, "e4m3", seed=2, k_scale=ks, v_scale=2.0 ** -6)
    sign = np.where(np.arange(96 + n) % 2 == 0, 1.0, -1.0)
    k = torch.zeros((96 + n, 2, D), dtype=torch.float64)
    k[:, :, 3] = k[:, :, D - 7] = torch.from_numpy(2.0 ** -6 * sign)[:, None]
    _set_rows(pb, 0, k)
    _set_rows(pb, 1, torch.from_numpy(64.0 * sign)[:, None, None].expand(96 + n, 2, D))
    q = torch.zeros((n, 4, D), dtype=torch.float64)
    q[:, :, 3], q[:, :, D - 7] = 249 * 2.0 ** 120, -223 * 2.0 ** 120
    q = q.bfloat16()
    parents = np.arange(-1, n - 1).astype(np.int32)
    scale = 0.5 / (26 * 2.0 ** 114 * ks)
    got = _run_attention(pb, q.cuda(), parents, scale).cpu().double()
    O, _, S = _attention64(pb, q, parents, scale)
    # as above, without a rounding of q: every value has 8 bits
    delta = (2 * (D + 2) * F32_HALF * S)[..., None]
    lim = BF16_HALF * O.abs() + (1 - O * O) * delta + delta ** 2 + F16_HALF + 1024 * F32_HALF
    off = (got - O).abs()
    assert (off <= lim).all(), (off / lim).max()


# ---- factors on the scores at the ends of FP32 ------------------------------------

@pytest.mark.parametrize("n", [1, 12, 80])
def test_score_factors_below_fp32(n):
    """scale * k_scale below FP32's smallest number: every visible position weighs
    the same, and masked ones nothing.  The same where a row of q makes it so."""
    keys = 20 * torch.from_numpy(np.random.default_rng(n).standard_normal((100 + n, 2, 128)))
    for k_scale, scale, q_scale in ((1e-30, 1e-20, 2.0), (1e-12, 0.0, 1e-34), (1.0, 1e-45, 2.0)):
        dtype = "bf16" if k_scale == 1.0 else "e4m3"
        pb = Problem([100], [n], 2, 128, 16, dtype, k_scale=k_scale)
        _set_rows(pb, 0, keys.float().to(pb.K.dtype).float())
        got = _check_attention(pb, 8, "star", scale=scale, q_scale=q_scale)
        assert torch.isfinite(got.float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 12, 80])
def test_score_factors_above_fp32(n, dtype):
    """scale * log2(e) * k_scale past FP32's largest number, and keys of zero: all
    scores are 0."""
    pb = Problem([100], [n], 2, 128, 16, dtype, k_scale=1e10)
    _set_rows(pb, 0, torch.zeros((100 + n, 2, 128)))
    assert torch.isfinite(_check_attention(pb, 8, "tree", scale=3e38).float()).all()
    if dtype == "e4m3":
        _check_attention(pb, 8, "tree", scale=1e20, q_scale=1e37)


# ---- lengths that change between calls in flight -----------------------------------

@pytest.mark.parametrize("n", [1, 3, 12])
@pytest.mark.parametrize("B", [3, 40, 300])
def test_lengths_written_right_before_the_call(B, n):
    """Calls back to back on one stream, each behind a kernel that writes its
    lengths (and, every other time, ranges): both kernels of a call see those."""
    rng = np.random.default_rng(B + n)
    pb = Problem([400 if B < 100 else 60] * B, [n] * B, 2, 64, 16, seed=B)
    q = torch.from_numpy(rng.standard_normal((pb.N, 8, 64))).bfloat16().cuda()
    ws = torch.empty(Q.qmm_tree_attention_workspace_bytes(pb.cache, 8, n), dtype=torch.uint8,
                     device="cuda")
    d_lens, d_cu = torch.zeros_like(pb.d_lens), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cache = Q.kv_cache(pb.K, pb.V, pb.d_table, d_lens)
    # one token a sequence and no child: accept writes new_lens = lens + 1
    one = torch.zeros(B, dtype=torch.int32, device="cuda")
    path, count = torch.zeros((B, 1), dtype=torch.int32, device="cuda"), torch.zeros_like(one)
    sets = []
    for _ in range(5):
        base = _dev(rng.integers(0, pb.lens[0], B).astype(np.int32))
        sets.append((base, Q.kv_caches([Q.kv_cache(pb.K, pb.V, pb.d_table, base)]),
                     _dev(np.concatenate([[0], np.cumsum(rng.integers(0, n + 1, B))]).astype(np.int32))))

    def call(i, O):
        base, caches, cu = sets[i % 5]
        if i % 2:
            d_cu.copy_(cu)
        Q.qmm_tree_accept(caches, one, one, 1, path, count, new_lens=d_lens)
        Q.qmm_tree_attention(cache, q, O, n, cu=d_cu if i % 2 else None, workspace=ws)

    want = [torch.full_like(q, 7.0) for _ in range(10)]
    for i, O in enumerate(want):
        call(i, O)
        torch.cuda.synchronize()
        assert torch.equal(d_lens, sets[i % 5][0] + 1)
    got = [torch.full_like(q, 7.0) for _ in range(200)]
    torch.cuda.synchronize()
    for i, O in enumerate(got):
        call(i, O)
    torch.cuda.synchronize()
    for i, O in enumerate(got):
        assert torch.equal(O.view(torch.int16), want[i % 10].view(torch.int16)), i


# ---- append in place -------------------------------------------------------------

@pytest.mark.parametrize("N,Hq,Hkv,D", [(5, 8, 2, 128), (700, 8, 2, 64), (900, 200, 4, 128),
                                        (300, 333, 1, 64)])
def test_append_in_place_equals_out_of_place(N, Hq, Hkv, D):
    """q_out = q, from fewer heads than a lane group holds at once to many times
    that: the same q and the same cache as with an output of its own."""
    rng = np.random.default_rng(N)
    x = torch.from_numpy(rng.standard_normal((N, Hq + 2 * Hkv, D))).bfloat16().cuda()
    ang = np.arange(N)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)
    cs = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float().cuda()
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).bfloat16().cuda()
    rope = Q.rope(cs, q_norm=w, k_norm=w)
    got = []
    for in_place in (False, True):
        pages = -(-N // 16)
        pools = [torch.zeros((pages, Hkv, 16, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        cache = Q.kv_cache(*pools, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
                           torch.zeros(1, dtype=torch.int32, device="cuda"))
        y = x.clone()
        out = y[:, :Hq] if in_place else torch.empty((N, Hq, D), dtype=torch.bfloat16, device="cuda")
        Q.qmm_kv_append(cache, y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], out, rope=rope)
        assert torch.equal(y[:, Hq:], x[:, Hq:]) and (in_place or torch.equal(y, x))
        got.append([t.contiguous().view(torch.int16) for t in (out, *pools)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ---- memory around the buffers ----------------------------------------------------

class Guarded:
    """Buffers of exact size inside larger ones whose rest holds a pattern."""
    PAD = 1 << 16

    def __init__(self):
        self.all = []

    def like(self, t, fill=None):
        """A copy of t (or its shape and type, filled) with guards on both sides."""
        n = t.numel() * t.element_size()
        raw = torch.full((n + 2 * self.PAD,), 0xA5, dtype=torch.uint8, device="cuda")
        view = raw[self.PAD:self.PAD + n].view(t.dtype).view(t.shape)
        view.copy_(t) if fill is None else view.fill_(fill)
        self.all.append((raw, n))
        return view

    def check(self):
        torch.cuda.synchronize()
        for raw, n in self.all:
            assert (raw[:self.PAD] == 0xA5).all() and (raw[self.PAD + n:] == 0xA5).all()


def _guarded_cache(pb, g):
    """pb's cache with guards around its pools, table and lengths."""
    nhd = pb.K.stride(2) > pb.K.stride(1)
    pools = []
    for t in (pb.K, pb.V):
        base = t.transpose(1, 2) if nhd else t
        assert base.is_contiguous()
        base = g.like(base.view(torch.uint8)).view(t.dtype).view(base.shape)
        pools.append(base.transpose(1, 2) if nhd else base)
    return pools, Q.kv_cache(*pools, g.like(pb.d_table), g.like(pb.d_lens), *pb.scales)


@pytest.mark.parametrize("cu", [[0, 99, 3, 12], [0, 4, 8, 2 ** 31 - 1], [12, 8, 4, 0],
                                [0, 12, 12, 12], [3, 5, 5, 9], [-5, 4, 8, 12],
                                [-2 ** 31, -2 ** 31, 2, 30]])
@pytest.mark.parametrize("T", [4, 12])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_ranges_out_of_order_write_only_their_rows(cu, T, dtype):
    """cu is device data: its values are clamped.  Rows of no range, slots of no
    token and everything around the buffers stay as they were."""
    pb = Problem([30, 14, 47], [4, 4, 4], 2, 64, 16, dtype)
    N, g = 12, Guarded()
    (K, V), cache = _guarded_cache(pb, g)
    d_cu = g.like(_dev(np.array(cu, np.int64).astype(np.int32)))
    q = g.like(torch.randn((N, 8, 64), device="cuda").bfloat16())
    O, q_out = g.like(q, 7.0), g.like(q, 7.0)
    k, v = (g.like(torch.randn((N, 2, 64), device="cuda").bfloat16()) for _ in range(2))
    nb = Q.qmm_tree_attention_workspace_bytes(cache, 8, T)
    ws = g.like(torch.empty(nb, dtype=torch.uint8, device="cuda"), 0xFF)
    bits = torch.int8 if dtype == "e4m3" else torch.int16
    old = [t.contiguous().view(bits).clone() for t in (K, V)]
    Q.qmm_tree_attention(cache, q, O, T, cu=d_cu, workspace=ws)
    g.check()
    rows = set()
    for b in range(3):
        a = min(max(cu[b], 0), N)
        e = min(max(cu[b + 1], a), N)
        rows |= set(range(a, min(e, a + T)))
    for r in range(N):
        assert bool((O[r] == 7.0).all()) == (r not in rows), r
    assert all(torch.equal(t.contiguous().view(bits), o) for t, o in zip((K, V), old))
    Q.qmm_kv_append(cache, q, k, v, q_out, cu=d_cu)
    g.check()
    want = [o.clone() for o in old]
    written = set()
    for t in range(N):
        b = sum(c <= t for c in cu[1:])
        if b < 3 and t >= cu[b]:
            written.add(t)
            s = pb.lens[b] + t - max(cu[b], 0)
            if s < pb.width * 16 and 0 <= pb.table[b, s // 16] < K.shape[0]:
                for w, x, pool, sc in zip(want, (k, v), (K, V), pb.scales):
                    y = (x[t].float() / sc).clamp(-448, 448) if dtype == "e4m3" else x[t]
                    w[int(pb.table[b, s // 16]), :, s % 16] = y.to(pool.dtype).view(bits)
    for r in range(N):
        assert torch.equal(q_out[r], q[r]) if r in written else (q_out[r] == 7.0).all(), r
    assert all(torch.equal(t.contiguous().view(bits), w) for t, w in zip((K, V), want))


@pytest.mark.parametrize("lens,n,Hq,Hkv,D,page,dtype,layout", [
    ([70, 3], [1, 1], 8, 2, 128, 16, "bf16", "hnd"),
    ([70, 3], [2, 2], 8, 2, 64, 8, "e4m3", "nhd"),
    ([70, 0, 9], [5, 0, 9], 6, 2, 128, 16, "bf16", "nhd"),
    ([70, 0, 9], [5, 0, 9], 6, 2, 128, 64, "e4m3", "hnd"),
    ([300, 64], [70, 90], 9, 3, 64, 32, "bf16", "hnd"),
    ([300, 64], [70, 90], 9, 3, 128, 32, "e4m3", "nhd"),
    ([3000], [256], 8, 1, 128, 16, "bf16", "hnd"),
])
def test_a_step_between_guards(lens, n, Hq, Hkv, D, page, dtype, layout):
    """Append, attention and accept with every buffer of exactly its size."""
    pb, g = Problem(lens, n, Hkv, D, page, dtype, layout, spare=0, width=None), Guarded()
    rng = np.random.default_rng(len(lens))
    (K, V), cache = _guarded_cache(pb, g)
    N, B, T = pb.N, pb.B, pb.T
    cu = None if pb.uniform else g.like(_dev(pb.cu))
    q = g.like(torch.randn((N, Hq, D), device="cuda").bfloat16())
    k, v = (g.like(torch.randn((N, Hkv, D), device="cuda").bfloat16()) for _ in range(2))
    q_out, O = g.like(q, 7.0), g.like(q, float("nan"))
    rows = max(lens) + max(n)
    ang = np.arange(rows)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)
    cs = g.like(torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float())
    w = g.like(torch.ones(D, device="cuda").bfloat16())
    pos = g.like(_dev(np.concatenate([a + np.arange(m) for a, m in zip(lens, n)]).astype(np.int32)))
    par = g.like(_dev(np.concatenate([_tree(rng, m, "tree") for m in n]).astype(np.int32)))
    tok, tgt = (g.like(_dev(rng.integers(0, 2, N).astype(np.int32))) for _ in range(2))
    ws = g.like(torch.empty(Q.qmm_tree_attention_workspace_bytes(cache, Hq, T), dtype=torch.uint8,
                            device="cuda"), 0xFF)
    path = g.like(torch.empty((B, T), dtype=torch.int32, device="cuda"), 99)
    count, nxt, new = (g.like(torch.empty(B, dtype=torch.int32, device="cuda"), 99) for _ in range(3))
    before = [t.clone() for t in (q, k, v, cs, w, pos, par, tok, tgt)]
    Q.qmm_kv_append(cache, q, k, v, q_out, rope=Q.rope(cs, q_norm=w, k_norm=w), positions=pos, cu=cu)
    Q.qmm_tree_attention(cache, q_out, O, T, parents=par, cu=cu, workspace=ws)
    Q.qmm_tree_accept(Q.kv_caches([cache]), tok, tgt, T, path, count, nxt, new, parents=par, cu=cu)
    g.check()
    assert torch.isfinite(O.float()).all() and not (q_out == 7.0).all(-1).any()
    assert all(torch.equal(a, b) for a, b in zip(before, (q, k, v, cs, w, pos, par, tok, tgt)))
    for t in (path, count, nxt, new):
        assert not (t == 99).any()


def test_strides_of_one_row_may_differ_between_k_and_v():
    """One page of one head: only the strides of the slots have to agree."""
    pb = Problem([3], [4], 1, 128, 8, spare=0, width=1)
    want = _check_attention(pb, 2)
    V = pb.V.as_strided((1, 1, 8, 128), (8, 24, 128, 1))
    pb.cache = Q.kv_cache(pb.K, V, pb.d_table, pb.d_lens)
    assert torch.equal(_check_attention(pb, 2).view(torch.int16), want.view(torch.int16))
    wide = torch.zeros((1, 1, 8, 256), dtype=torch.bfloat16, device="cuda")[..., :128]
    with pytest.raises(ValueError, match="equal strides"):
        Q.kv_cache(pb.K, wide, pb.d_table, pb.d_lens)
