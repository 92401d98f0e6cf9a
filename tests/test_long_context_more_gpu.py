"""The paged cache's long-context calls on a GB300 at the borders of their sizes and their
memory."""
import math

import numpy as np
import pytest
import torch

from split_w4a16_quantized_gb300 import qmm as Q
from test_long_context_gpu import Shared, _check_prefix, _check_scored, _kept, _run_prefix, \
    _run_scored, _same, _scored64, _within
from test_paged_gpu import F32_HALF, Problem, _cos_sin, _dev, _tree
from test_paged_more_gpu import Guarded, _guarded_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    yield
    torch.cuda.synchronize()
    assert Q.qmm_kernel_status(clear=True) == 0


@pytest.mark.parametrize("lens,n,Hq,Hkv,D,page,dtype,layout", [
    ([70, 3], [1, 1], 8, 2, 128, 16, "bf16", "hnd"),
    ([70, 3], [2, 2], 8, 2, 64, 8, "e4m3", "nhd"),
    ([70, 0, 9], [5, 0, 9], 6, 2, 128, 16, "bf16", "nhd"),
    ([70, 0, 9], [5, 0, 9], 6, 2, 128, 64, "e4m3", "hnd"),
    ([300, 64], [70, 90], 9, 3, 64, 32, "bf16", "hnd"),
    ([300, 64], [70, 90], 9, 3, 128, 32, "e4m3", "nhd"),
    ([3000], [256], 8, 1, 128, 16, "bf16", "hnd"),
])
def test_every_call_between_guards(lens, n, Hq, Hkv, D, page, dtype, layout):
    """Append, both attentions and eviction with every buffer of exactly its size."""
    pb, g = Problem(lens, n, Hkv, D, page, dtype, layout, spare=0), Guarded()
    pb.table = pb.table[:, :max(-(-(a + b) // page) for a, b in zip(lens, n))].copy()
    pb.width = pb.table.shape[1]
    pb.bind()
    (K, V), cache = _guarded_cache(pb, g)
    N, B, T = pb.N, pb.B, pb.T
    cu = None if pb.uniform else g.like(_dev(pb.cu))
    q = g.like(torch.randn((N, Hq, D), device="cuda").bfloat16())
    k, v = (g.like(torch.randn((N, Hkv, D), device="cuda").bfloat16()) for _ in range(2))
    q_out, O, O2 = g.like(q, 7.0), g.like(q, float("nan")), g.like(q, float("nan"))
    cs, pos = g.like(_cos_sin(50, D)), g.like(torch.randint(0, 50, (3, N), dtype=torch.int32))
    Q.qmm_kv_append_axes(cache, q, k, v, pos, Q.rope_axes([j % 3 for j in range(D // 2)]),
                         Q.rope(cs), q_out=q_out, cu=cu)
    # the first sequence's table is the prefix of all but the last
    prefix = Q.prefix(g.like(_dev(pb.table[:1])), g.like(_dev(np.array([lens[0]], np.int32))),
                      g.like(_dev(np.array([0, max(1, B - 1)], np.int32))))
    nb = Q.qmm_prefix_attention_workspace_bytes(cache, Hq, N, T)
    ws = g.like(torch.empty(nb, dtype=torch.uint8, device="cuda"), 0xFF)
    par = g.like(_dev(np.concatenate([_tree(np.random.default_rng(b), m, "tree")
                                      for b, m in enumerate(n)]).astype(np.int32)))
    Q.qmm_prefix_attention(cache, prefix, q_out, O, T, parents=par, cu=cu, workspace=ws)
    S = pb.width * page
    mass = g.like(torch.zeros((1, B, Hkv, S), device="cuda"))
    nb = Q.qmm_scored_attention_workspace_bytes(cache, Hq, T)
    ws2 = g.like(torch.empty(nb, dtype=torch.uint8, device="cuda"), 0xFF)
    Q.qmm_scored_attention(cache, q_out, O2, T, mass, cu=cu, workspace=ws2)
    kept = g.like(torch.empty((1, B, Hkv, 20), dtype=torch.int32, device="cuda"), -7)
    new = g.like(torch.empty(B, dtype=torch.int32, device="cuda"), -7)
    out = g.like(mass, 9.0)
    Q.qmm_kv_evict(Q.kv_caches([cache]), mass, 20, kept, new, sinks=1, recent=5, mass_out=out)
    g.check()
    for o in (O, O2):
        assert torch.isfinite(o.float()).all()
    assert torch.isfinite(mass).all() and not (q_out == 7.0).all(-1).any()
    assert not (kept == -7).any() and not (new == -7).any()


def _far(pb, pages):
    """pb's pages at both ends of pools of so many: the pools and the table."""
    ids = [pages - 1 - i if i % 3 else i for i in range(pb.K.shape[0])]
    pools = []
    for src in (pb.K, pb.V):
        pool = torch.empty((pages, *src.shape[1:]), dtype=src.dtype, device="cuda")
        pool.view(torch.int16)[ids] = src.view(torch.int16)
        pools.append(pool)
    table = np.where(pb.table >= 0, np.asarray(ids)[np.clip(pb.table, 0, None)], -1).astype(np.int32)
    return pools, table, ids


@pytest.mark.parametrize("n", [1, 30])
def test_pools_beyond_32_bits(n):
    """Pages whose offsets pass 2^32 bytes and 2^31 values: the same bits."""
    free, _ = torch.cuda.mem_get_info()
    if free < 16 << 30:
        pytest.skip("needs 11 GB")
    Hkv, page, D = 8, 64, 128
    pb = Problem([190, 70, 300], [n, n, 0], Hkv, D, page, seed=8)
    (K, V), table, ids = _far(pb, 40000)
    q = torch.randn((2 * n, 32, D), device="cuda").bfloat16()
    S = pb.width * page
    weights = torch.rand((1, 2, Hkv, S), device="cuda")
    got = []
    for k, v, t in ((pb.K, pb.V, pb.table), (K, V, table)):
        lens = _dev(np.array([190, 70], np.int32))
        cache = Q.kv_cache(k, v, _dev(t[:2]), lens)
        pre = Q.prefix(_dev(t[2:]), _dev(np.array([300], np.int32)), _dev(np.array([0, 2], np.int32)))
        O, O2, mass = torch.empty_like(q), torch.empty_like(q), torch.ones((2, Hkv, S), device="cuda")
        ws = torch.empty(max(Q.qmm_prefix_attention_workspace_bytes(cache, 32, 2 * n, n),
                             Q.qmm_scored_attention_workspace_bytes(cache, 32, n)),
                         dtype=torch.uint8, device="cuda")
        Q.qmm_prefix_attention(cache, pre, q, O, n, workspace=ws)
        Q.qmm_scored_attention(cache, q, O2, n, mass, workspace=ws)
        kept = torch.empty((1, 2, Hkv, 40), dtype=torch.int32, device="cuda")
        out = torch.zeros_like(weights)
        Q.qmm_kv_evict(Q.kv_caches([cache]), weights, 40, kept, _dev(np.zeros(2, np.int32)),
                       sinks=1, recent=9, mass_out=out)
        x = torch.randn((2 * n, 2 * Hkv, D), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
        Q.qmm_kv_append_axes(cache, None, x[:, :Hkv].bfloat16(), x[:, Hkv:].bfloat16(),
                             _dev(np.full((2, 2 * n), 3, np.int32)), Q.rope_axes([0, 1] * 32),
                             Q.rope(_cos_sin(9, D).cuda()))
        got.append([O, O2, mass, kept, out] + [p[ids] if p.shape[0] == 40000 else p for p in (k, v)])
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert _same(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_thousands_of_sequences(dtype):
    rng = np.random.default_rng(2)
    lens = [int(v) for v in rng.integers(0, 40, 3001)]
    _check_scored(Problem(lens, [1] * 3001, 1, 64, 8, dtype, seed=4), 4)
    first = np.sort(rng.integers(0, 3002, 400)).tolist()
    _check_prefix(Shared([int(v) for v in rng.integers(0, 30, 399)], first, lens, [1] * 3001, 1, 64, 8,
                         dtype, seed=4), 4, "chain")


def test_most_rows_of_a_prefix():
    """More query rows of one prefix than 2^14, tokens of 256 a sequence."""
    _check_prefix(Shared([130], [0, 9], [3, 0, 9, 1, 5, 64, 2, 2, 2], [256] * 9, 1, 64, 16), 8, "star")


def test_prefix_with_most_heads_to_a_group():
    _check_prefix(Shared([70], [0, 3], [3, 0, 9], [100, 3, 7], 1, 128, 16, "e4m3"), 64)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_most_rows_of_scores(dtype):
    """Blocks of 256 rows that add to the same slots one after the other: 64 of them, the
    last in part."""
    _check_scored(Problem([140], [255], 1, 64, 16, dtype), 64, 0.5)
    _check_scored(Problem([140, 3], [33, 9], 2, 64, 16, dtype), 32, 0.0)


@pytest.mark.parametrize("n", [3, 30])
def test_scored_past_the_table(n):
    """Cached tokens up to the table's end: the new ones have no slots, and give their
    weight to the cached ones."""
    pb = Problem([64, 64], [0, 0], 2, 128, 16, width=4)
    pb.n, pb.cu, pb.N, pb.T = [n, n], np.array([0, n, 2 * n], np.int32), 2 * n, n
    pb.uniform = True
    q = torch.randn((2 * n, 8, 128), device="cuda").bfloat16()
    mass = torch.zeros((2, 2, 64), device="cuda")
    _run_scored(pb, q, mass, 1.0)
    m = mass.cpu()
    for b in range(2):
        s = torch.einsum("nhgd,lhd->nhgl", q.cpu()[b * n:b * n + n].double().view(n, 2, 4, 128),
                         pb.values[0][b]) / math.sqrt(128)
        want = s.softmax(-1).sum((0, 2))
        # scores and sums in FP32: (D + 2) 2^-24 of sum |q k| < 30, twice, and the sums
        assert ((m[b].double() - want).abs() <= 2.0 ** -11 * want + 1e-30).all()
    pb.lens = [2 ** 31 - 1, -7]          # clamped: the whole table, nothing
    pb.bind()
    again = torch.zeros((2, 2, 64), device="cuda")
    _run_scored(pb, q, again, 1.0)
    assert _same(again[0], mass[0])
    assert (again[1, :, min(n, 64):] == 0).all() and torch.isfinite(again).all()


@pytest.mark.parametrize("n", [1, 20])
def test_scored_sequences_without_tokens_fade(n):
    """decay of a sequence's sums, whether it has tokens or not."""
    pb = Problem([50, 1500, 9], [n, 0, n], 2, 64, 16)
    _, mass = _check_scored(pb, 8, 0.5)
    assert mass.shape[0] == 3


def test_scored_steps_add_up():
    """Steps one after the other give what their sum is, and a graph of them too."""
    pb = Problem([200, 31], [1, 1], 2, 128, 16)
    qs = [torch.randn((2, 8, 128), device="cuda").bfloat16() for _ in range(4)]
    parts = []
    for q in qs:
        m = torch.zeros((2, 2, pb.width * 16), device="cuda")
        _run_scored(pb, q, m, 0.0)
        parts.append(m.double())
    total, O = torch.zeros((2, 2, pb.width * 16), device="cuda"), torch.empty_like(qs[0])
    ws = torch.empty(Q.qmm_scored_attention_workspace_bytes(pb.cache, 8, 1), dtype=torch.uint8,
                     device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for q in qs:
            Q.qmm_scored_attention(pb.cache, q, O, 1, total, workspace=ws)
    total.zero_()
    g.replay()
    torch.cuda.synchronize()
    for b, ln in enumerate((200, 31)):
        want = sum(p[b] for p in parts)
        want[:, ln] = parts[-1][b][:, ln]     # the new token's slot starts again each time
        assert ((total[b].double() - want).abs()[:, :ln + 1] <=
                8 * F32_HALF * want[:, :ln + 1]).all()


def test_evict_budgets_beyond_the_table_and_many_sequences():
    rng = np.random.default_rng(0)
    B, page = 700, 8
    lens = rng.integers(0, 33, B).astype(np.int32)
    K = torch.from_numpy(rng.integers(0, 60000, (B * 4, 1, page, 64)).astype(np.int32)).to(torch.int16)
    K = K.view(torch.bfloat16).cuda()
    V = K.clone()
    table = _dev(rng.permutation(B * 4).reshape(B, 4).astype(np.int32))
    cache = Q.kv_caches([Q.kv_cache(K, V, table, _dev(lens))])
    mass = torch.rand((B, 1, 32), device="cuda")
    old = K.view(torch.int16).clone()
    kept = torch.zeros((1, B, 1, 1000), dtype=torch.int32, device="cuda")
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    before = mass.clone()
    Q.qmm_kv_evict(cache, mass, 1000, kept, new, sinks=500, recent=500)   # more than there are
    assert new.tolist() == np.minimum(lens, 32).tolist() and _same(mass, before)
    assert torch.equal(K.view(torch.int16), old)
    assert ((kept[0, :, 0] >= 0).sum(-1).cpu().numpy() == np.minimum(lens, 32)).all()
    kept = torch.zeros((1, B, 1, 10), dtype=torch.int32, device="cuda")
    Q.qmm_kv_evict(cache, mass, 10, kept, new, sinks=2, recent=3)
    for b in range(0, B, 7):
        k = _kept(before[b, 0].cpu().numpy(), min(int(lens[b]), 32), 10, 2, 3)
        assert kept[0, b, 0, :len(k)].tolist() == k.tolist()
        for j, s in enumerate(k):
            at = [(int(table[b, i // page]), 0, i % page) for i in (int(j), int(s))]
            assert torch.equal(K.view(torch.int16)[at[0]], old[at[1]])


@pytest.mark.parametrize("lens,keep,again,Hkv", [
    ([40000, 20001], 9000, 3000, 1),     # a column shared by blocks, and its moves
    ([150000], 20000, 700, 1),           # more than the blocks of a column hold
    ([5000, 1, 3300], 2500, 600, 2),
])
def test_evictions_in_a_row_captured_and_replayed(lens, keep, again, Hkv):
    """Two evictions, the second of what the first left, in place and in one graph, replayed
    on a stream of its own with other weights and lengths: what single calls leave."""
    B, page, D = len(lens), 64, 64
    width = -(-max(lens) // page)
    g = torch.Generator(device="cuda").manual_seed(5)
    K0, V0 = (torch.randint(-2 ** 15, 2 ** 15, (B * width, Hkv, page, D), generator=g, device="cuda",
                            dtype=torch.int16) for _ in "kv")
    table = torch.randperm(B * width, generator=g, device="cuda").int().view(B, width)

    def state():
        K, V = K0.clone(), V0.clone()
        d_lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        mid, new = torch.zeros_like(d_lens), torch.zeros_like(d_lens)
        mass = torch.zeros((B, Hkv, width * page), device="cuda")
        kept = [torch.zeros((1, B, Hkv, k), dtype=torch.int32, device="cuda") for k in (keep, again)]
        caches = [Q.kv_caches([Q.kv_cache(K.view(torch.bfloat16), V.view(torch.bfloat16), table, x)])
                  for x in (d_lens, mid)]
        return dict(K=K, V=V, lens=d_lens, mid=mid, new=new, mass=mass, kept=kept, caches=caches)

    def load(st, ln, seed):
        w = torch.Generator(device="cuda").manual_seed(seed)
        st["lens"].copy_(torch.tensor(ln, dtype=torch.int32))
        st["mass"].copy_(torch.rand(st["mass"].shape, generator=w, device="cuda"))
        st["K"].copy_(K0), st["V"].copy_(V0)

    def call(st, i):
        Q.qmm_kv_evict(st["caches"][i], st["mass"], (keep, again)[i], st["kept"][i],
                       st[("mid", "new")[i]], sinks=4, recent=200)

    graphed, single = state(), state()
    load(graphed, lens, 1)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(graphed, 0), call(graphed, 1)
    for seed, ln in ((2, lens), (3, [x // 2 for x in lens]), (4, [min(x, keep) for x in lens])):
        load(graphed, ln, seed), load(single, ln, seed)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            call(single, i)
            torch.cuda.synchronize()
        for name in ("K", "V", "mid", "new"):
            assert torch.equal(graphed[name], single[name])
        assert _same(graphed["mass"], single["mass"])
        assert all(torch.equal(x, y) for x, y in zip(graphed["kept"], single["kept"]))
        w = torch.rand(graphed["mass"].shape, generator=torch.Generator(device="cuda").manual_seed(seed),
                       device="cuda").cpu().numpy()
        for b, x in enumerate(ln):   # and the first of the two is the formula's
            for h in range(Hkv):
                k = _kept(w[b, h], x, keep, 4, 200)
                assert graphed["kept"][0][0, b, h, :len(k)].tolist() == k.tolist()


def test_attention_is_the_same_behind_an_eviction():
    """The order of the kept slots changes nothing but the order of sums: attention over the
    evicted cache is attention over the kept rows."""
    pb = Problem([400, 90], [0, 0], 2, 128, 16, seed=6)
    mass = torch.rand((1, 2, 2, pb.width * 16), device="cuda")
    weights = mass.cpu().numpy()
    kept = torch.zeros((1, 2, 2, 80), dtype=torch.int32, device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    Q.qmm_kv_evict(Q.kv_caches([pb.cache]), mass, 80, kept, new, sinks=4, recent=16)
    for b in range(2):
        for i in range(2):
            rows = pb.values[i][b]
            pb.values[i][b] = torch.stack(
                [rows[_kept(weights[0, b, h], pb.lens[b], 80, 4, 16), h] for h in range(2)], 1)
    pb.lens = [80, 80]
    pb.n, pb.cu, pb.N, pb.T, pb.uniform = [1, 1], np.array([0, 1, 2], np.int32), 2, 1, True
    # one more token each, appended behind the budget
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((2, 4, 128))).bfloat16()
    pb.bind()
    Q.qmm_kv_append(pb.cache, None, x[:, :2].cuda(), x[:, 2:].cuda())
    for b in range(2):
        for i in range(2):
            pb.values[i][b] = torch.cat([pb.values[i][b], x[b:b + 1, 2 * i:2 * i + 2].double()])
    _check_scored(pb, 8, 1.0)


@pytest.mark.parametrize("B", [1, 8, 40, 300])
@pytest.mark.parametrize("n", [1, 3, 24])
def test_lengths_written_right_before_the_calls(B, n):
    """The launches of a call plan from lens, the first without waiting for anything but
    what comes before it: lengths and prefixes written by the kernel just before."""
    sh = Shared([150], [0, B], [40] * B, [n] * B, 1, 64, 16, seed=B)
    q = torch.randn((B * n, 4, 64), device="cuda").bfloat16()
    ws = torch.empty(max(Q.qmm_prefix_attention_workspace_bytes(sh.cache, 4, B * n, n),
                         Q.qmm_scored_attention_workspace_bytes(sh.cache, 4, n)),
                     dtype=torch.uint8, device="cuda")
    S = sh.cache.max_pages * 16
    lens = [sh.d_lens.clone(), torch.randint(0, 41, (B,), dtype=torch.int32, device="cuda")]
    plens = [sh.d_plens.clone(), torch.full_like(sh.d_plens, 37)]
    want = []
    for ln, pl in zip(lens, plens):
        sh.d_lens.copy_(ln), sh.d_plens.copy_(pl)
        torch.cuda.synchronize()
        O, O2, m = torch.zeros_like(q), torch.zeros_like(q), torch.ones((B, 1, S), device="cuda")
        Q.qmm_prefix_attention(sh.cache, sh.prefix, q, O, n, workspace=ws)
        Q.qmm_scored_attention(sh.cache, q, O2, n, m, workspace=ws)
        want.append((O, O2, m))
    torch.cuda.synchronize()
    assert not _same(want[0][0], want[1][0])
    big = torch.empty(1 << 26, device="cuda")
    for i in range(12):
        O, O2, m = torch.zeros_like(q), torch.zeros_like(q), torch.ones((B, 1, S), device="cuda")
        big.fill_(i)
        sh.d_lens.copy_(lens[i % 2]), sh.d_plens.copy_(plens[i % 2])
        Q.qmm_prefix_attention(sh.cache, sh.prefix, q, O, n, workspace=ws)
        Q.qmm_scored_attention(sh.cache, q, O2, n, m, workspace=ws)
        for a, b in zip(want[i % 2], (O, O2, m)):
            assert _same(a, b)


def test_prefix_rows_on_both_sides_of_the_kernels():
    """16 query rows in all and more; 8 of a sequence and more."""
    for B, n, Hq in ((4, 1, 8), (5, 1, 8), (2, 2, 8), (3, 2, 8), (1, 3, 6), (2, 1, 32), (2, 9, 2),
                     (1, 8, 2), (1, 9, 2), (16, 1, 2), (17, 1, 2)):
        for dtype in ("bf16", "e4m3"):
            _check_prefix(Shared([77], [0, B], [9 * b for b in range(B)], [n] * B, 2, 128, 16, dtype), Hq)


def test_prefix_values_that_are_not_numbers_stay_in_their_rows():
    for n, Hq in ((1, 8), (12, 16)):
        sh = Shared([130], [0, 2], [5, 40], [n, n], 2, 128, 16)
        q = torch.randn((2 * n, Hq, 128), device="cuda").bfloat16()
        clean = _run_prefix(sh, q, None)
        bad = q.clone()
        bad[0, 1, 3], bad[n, 2, 9] = float("nan"), float("inf")
        got = _run_prefix(sh, bad, None)
        touched = torch.zeros((2 * n, Hq), dtype=torch.bool)
        touched[0, 1] = touched[n, 2] = True
        assert not torch.isfinite(got[touched].float()).any()
        assert _same(got[~touched], clean[~touched])


def test_scored_limits_of_the_window():
    """The window of a prompt: the weights of its own chain, token by token."""
    pb = Problem([0], [64], 1, 128, 16)
    q = torch.zeros((64, 2, 128), dtype=torch.bfloat16, device="cuda")
    mass = torch.full((1, 1, pb.width * 16), float("nan"), device="cuda")
    _run_scored(pb, q, mass, 1.0)
    # every score is 0: token i gives 1 / (i + 1) of each head's weight to slots 0 .. i
    want = torch.tensor([2 * sum(1 / (i + 1) for i in range(s, 64)) for s in range(64)]).double()
    _within(mass[0, 0, :64].cpu(), want, 200 * F32_HALF * want)
    assert torch.isnan(mass[0, 0, 64:]).all()
    O, A, S, W, E = _scored64(pb, q.cpu(), 1.0)
    assert (W[0][0] - want).abs().max() < 1e-5
