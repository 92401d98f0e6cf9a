"""The paged cache's long-context calls on a GB300: what their interface promises of bits,
of slots out of sight and of device data out of range."""
import math

import numpy as np
import pytest
import torch

from test_long_context_gpu import PREFIX, Shared, _check_prefix, _o_limit, _prefix64, _run_prefix, \
    _run_scored, _same, _within
from test_paged_gpu import BF16_HALF, F32_HALF, Problem, _dev, _tree
from split_w4a16_quantized_gb300 import qmm as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    yield
    torch.cuda.synchronize()
    assert Q.qmm_kernel_status(clear=True) == 0


# ---- shared prefixes -----------------------------------------------------------------

def _width(page, long):
    """Pages of a table: as many as are needed, or so many that a call of more than 8 rows
    takes the tcgen05 kernel."""
    return 8192 // page if long else None


@pytest.mark.parametrize("plens,first,lens,n,Hq,Hkv,D,page,dtype,layout,kind", PREFIX,
                         ids=["%d" % i for i in range(len(PREFIX))])
def test_prefix_of_long_tables(plens, first, lens, n, Hq, Hkv, D, page, dtype, layout, kind):
    _check_prefix(Shared(plens, first, lens, n, Hkv, D, page, dtype, layout, width=_width(page, True)),
                  Hq, kind)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 5])
def test_prefix_of_long_tables_many_sequences_and_groups(n, dtype):
    rng = np.random.default_rng(5)
    lens = [int(v) for v in rng.integers(0, 90, 300)]
    first = [0] + sorted(int(v) for v in rng.integers(0, 300, 39)) + [300]
    plens = [int(v) for v in rng.integers(0, 400, 40)]
    _check_prefix(Shared(plens, first, lens, [n] * 300, 1, 64, 16, dtype, seed=3, width=_width(16, True)), 4)


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("plens,first,lens,n,Hq,Hkv,D,page,layout,kind", [
    ([40], [0, 3], [5, 9, 0], [1] * 3, 8, 2, 128, 16, "hnd", "chain"),           # 12 rows
    ([40], [0, 12], list(range(12)), [1] * 12, 8, 2, 128, 16, "hnd", "chain"),   # 48
    ([50], [0, 40], [i % 9 for i in range(40)], [1] * 40, 16, 4, 64, 16, "nhd", "chain"),
    ([30, 61], [0, 5, 9], [5, 7, 0, 6, 3, 3, 4, 9, 1], [8] * 9, 16, 4, 128, 16, "nhd", "tree"),
    ([64], [1, 3], [5, 3, 0], [7, 9, 5], 8, 2, 64, 32, "hnd", "tree"),
], ids=["12", "48", "160", "groups", "ragged"])
def test_prefix_bf16_weights_have_two_terms(plens, first, lens, n, Hq, Hkv, D, page, layout, kind,
                                             long):
    """A BF16 cache's weights are two BF16 terms for any number of rows: the first is off by
    at most 2^-8 of the weight, the second by 2^-8 of that.  Beside it, as wholes of 2^-23
    (the tensor cores may cut where a sum would be rounded): scores of D products, in the
    weight and in their sum; sums over the positions; exp2 (2 ulp) and the divisions."""
    sh = Shared(plens, first, lens, n, Hkv, D, page, "bf16", layout, width=_width(page, long))
    rng = np.random.default_rng(7)
    q = torch.from_numpy(0.1 * rng.standard_normal((sh.N, Hq, D))).bfloat16()
    parents = np.concatenate([_tree(rng, m, kind) for m in n]).astype(np.int32)
    got = _run_prefix(sh, q.cuda(), None if kind == "chain" else parents)
    O, A, S = _prefix64(sh, q, parents, 1 / math.sqrt(D))
    positions = max(plens) + max(lens) + max(n)
    lim = BF16_HALF * O.abs() + A * (BF16_HALF ** 2 + 2 * F32_HALF * (
        2 * (D + 2) * S[..., None] + positions + 8)) + 1e-30
    _within(got.cpu(), O, lim)


# ---- weights by slot -----------------------------------------------------------------

@pytest.mark.parametrize("what", ["nan in q", "inf in q", "nan in k"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 2, 24])
def test_scored_not_numbers_stay_in_sight(n, dtype, what):
    """A row that is not a number leaves none in slots out of its sight, those of later
    tokens and those without a page, and all others of its sequence's head are; with few
    rows and with many."""
    pb = Problem([130, 5], [n, n], 2, 128, 16, dtype)
    pb.table[0, 2] = -1
    pb.bind()
    q = torch.randn((pb.N, 8, 128), device="cuda").bfloat16()
    old = torch.rand((2, 2, pb.width * 16), device="cuda")
    clean, mass = old.clone(), old.clone()
    _run_scored(pb, q, clean, 0.5)
    sees = torch.ones(130 + n, dtype=torch.bool)          # of slots, by the rows in question
    if what == "nan in k":
        # of the last token, which alone sees its own slot
        page, at = int(pb.table[0, (129 + n) // 16]), (129 + n) % 16
        pb.K.view(torch.uint8 if dtype == "e4m3" else torch.int16)[page, 0, at, 7] = \
            0x7f if dtype == "e4m3" else 0x7fc0
    else:
        q[0, 1, 5] = float(what[:3])
        sees[131:] = False
    _run_scored(pb, q, mass, 0.5)
    sees[32:48] = False
    assert _same(mass[1], clean[1]) and _same(mass[0, 1], clean[0, 1])
    got, want = mass[0, 0].cpu(), clean[0, 0].cpu()
    assert torch.isnan(got[:130 + n][sees]).all()
    assert _same(got[:130 + n][~sees], want[:130 + n][~sees])
    assert _same(got[130 + n:], want[130 + n:])
    assert _same(want[32:48], 0.5 * old[0, 0, 32:48].cpu())


def _seen(pools, table, slots, page):
    """K and V of a table's first slots in 64 bits, and which of them have pages."""
    pages = pools[0].shape[0]
    ids = torch.tensor([int(table[s // page]) for s in range(slots)], dtype=torch.int64)
    there = (ids >= 0) & (ids < pages)
    at = torch.arange(slots) % page
    return [p[ids.clamp(0, pages - 1), :, at].double() for p in pools], there


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq", [2, 8])      # 12 and 48 rows per KV head
@pytest.mark.parametrize("cu", [None, [0, 99, 3, 12, 12], [-5, 4, 8, 2 ** 31 - 1, 0],
                                [12, 8, 4, 0, 0], [0, 2, 5, 9, 2 ** 31 - 1]])
def test_prefix_of_clamped_device_values(cu, Hq, dtype):
    """first, lens and cu out of range count as clamped, for a sequence's rows and for those
    that see its prefix; rows of no sequence stay as they are."""
    N, T, B, D, page = 12, 3, 4, 64, 16
    sh = Shared([100, 50], [0, 2, 4], [30, 7, 3, 0], [T] * B, 2, D, page, dtype)
    pb, pools = sh.pb, []
    for pool, scale in zip((pb.K, pb.V), pb.scales):    # (slots that hold nothing: zeros)
        bits = pool.view(torch.uint8 if dtype == "e4m3" else torch.int16)
        bits[torch.isnan(pool.float())] = 0
        pools.append(pool.float().cpu() * scale)
    q = torch.randn((N, Hq, D)).bfloat16()
    ws = torch.empty(Q.qmm_prefix_attention_workspace_bytes(sh.cache, Hq, N, T), dtype=torch.uint8,
                     device="cuda")
    cap = pb.table.shape[1] * page
    tokens = np.arange(0, N + 1, T) if cu is None else np.clip(cu, 0, N)
    for first in ([-5, 2, 99], [4, 2, 0], [2 ** 31 - 1, -2 ** 31, 3], [1, 1, 1], [1, 3, 3]):
        for plens in ([100, 50], [-3, 2 ** 31 - 1], [0, 1]):
            sh.d_first.copy_(_dev(np.asarray(first, np.int32)))
            sh.d_plens.copy_(_dev(np.asarray(plens, np.int32)))
            O = torch.full((N, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
            Q.qmm_prefix_attention(sh.cache, sh.prefix, q.cuda(), O, T, workspace=ws,
                                   cu=None if cu is None else _dev(np.asarray(cu, np.int32)))
            want, A, S = (torch.zeros(s, dtype=torch.float64) for s in (O.shape, O.shape, O.shape[:2]))
            inside = torch.zeros(N, dtype=torch.bool)
            for b in range(B):
                start, end = int(tokens[b]), int(max(tokens[b], tokens[b + 1]))
                groups = [(min(max(first[g], 0), B), min(first[g + 1], B)) for g in range(2)]
                g = next((i for i, (lo, hi) in enumerate(groups) if lo <= b < hi), None)
                for i in range(min(end - start, T)):
                    r = start + i
                    inside[r] = True
                    parts = [(pb.table[b], sh.lens[b] + i + 1)]
                    if g is not None and tokens[groups[g][0]] <= r < tokens[groups[g][1]]:
                        parts.append((pb.table[B + g], min(max(plens[g], 0), cap)))
                    K, V, there = [], [], []
                    for table, slots in parts:
                        (k, v), t = _seen(pools, table, slots, page)
                        K.append(k), V.append(v), there.append(t)
                    there = torch.cat(there)
                    K, V = torch.cat(K)[there], torch.cat(V)[there]
                    x = q[r].double().view(2, -1, D)
                    p = (torch.einsum("hgd,lhd->hgl", x, K) / 8).softmax(-1)
                    want[r] = torch.einsum("hgl,lhd->hgd", p, V).reshape(Hq, D)
                    A[r] = torch.einsum("hgl,lhd->hgd", p, V.abs()).reshape(Hq, D)
                    S[r] = torch.einsum("hgd,lhd->hgl", x.abs(), K.abs()).amax(-1).reshape(Hq) / 8
            got = O.cpu()
            assert (got[~inside] == 7.0).all(), "a row of no sequence was written"
            _within(got[inside], want[inside], _o_limit(dtype == "e4m3", want, A, S, D)[inside])
