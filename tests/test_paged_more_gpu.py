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
