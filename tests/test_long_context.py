"""Shared prefixes, weights by slot, eviction and positions of several axes, host side
(CPU only): argument errors come back as codes before any CUDA work, workspace sizes,
and the binding's own checks."""
import ctypes

import pytest
import torch

from split_w4a16_quantized_gb300 import build
from split_w4a16_quantized_gb300 import qmm as Q
from test_paged import BAD_CACHES, PTR, _cache


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def _prefix_attend(cache, pre=None, q=PTR, qs=4096, O=PTR, N=8, T=2, Hq=32, cu=None, par=None,
                   scale=0.0, ws=PTR, nb=1 << 40, null=False, **kw):
    p = dict(table=PTR, lens=PTR, first=PTR, G=2, max_pages=30)
    p.update(kw)
    return Q.lib().qmm_prefix_attention(
        ctypes.byref(cache) if cache is not None else None,
        None if null else ctypes.byref(Q.qmm_prefix(**p)), q, qs, O, N, T, Hq, cu, par, scale, ws,
        nb, None)


def _scored(cache, q=PTR, qs=4096, O=PTR, N=8, T=2, Hq=32, cu=None, scale=0.0, mass=PTR, ms=320,
            decay=1.0, ws=PTR, nb=1 << 40):
    return Q.lib().qmm_scored_attention(ctypes.byref(cache) if cache is not None else None, q, qs,
                                        O, N, T, Hq, cu, scale, mass, ms, decay, ws, nb, None)


# B = 4, 8 heads, 320 slots, 2 layers, keep 16
def _evict(caches, n=None, mass=PTR, out=PTR, ls=4 * 8 * 320, ms=320, keep=16, sinks=2, recent=4,
           kept=2 << 20, new=3 << 20):
    arr = (Q.qmm_kv_cache * max(1, len(caches)))(*caches) if caches is not None else None
    return Q.lib().qmm_kv_evict(arr, n if n is not None else len(caches), mass, out, ls, ms, keep,
                                sinks, recent, kept, new, None)


def _axes(cache, q=PTR, k=PTR, v=PTR, out=PTR, N=8, Hq=32, qs=4096, ks=1024, vs=1024, os=4096,
          cu=None, pos=PTR, rope=True, axes=True, n=3, axis=None, **kw):
    r = dict(cos_sin=PTR, rows=100, dim=128, interleaved=0, eps=1e-6)
    r.update(kw)
    a = Q.qmm_rope_axes(n, (ctypes.c_uint8 * 64)(*(axis or [j % 3 for j in range(64)])))
    return Q.lib().qmm_kv_append_axes(
        ctypes.byref(cache) if cache is not None else None, q, k, v, out, N, Hq, qs, ks, vs, os,
        cu, pos, ctypes.byref(Q.qmm_rope(**r)) if rope else None,
        ctypes.byref(a) if axes else None, None)


@pytest.mark.parametrize("bad,code", BAD_CACHES, ids=[str(b[0]) for b in BAD_CACHES])
def test_bad_caches_refused_by_every_call(bad, code):
    c = _cache(**bad)
    assert _prefix_attend(c, cu=PTR) == code
    assert _scored(c, cu=PTR) == code
    assert _evict([_cache(), c] if code == Q.QMM_EINVAL else [c, c]) == code
    assert _axes(c, cu=PTR) == code
    L = Q.lib()
    assert L.qmm_prefix_attention_workspace_bytes(ctypes.byref(c), 32, 8, 2, 152) == 0
    assert L.qmm_scored_attention_workspace_bytes(ctypes.byref(c), 32, 2, 152) == 0


def test_null_caches():
    assert _prefix_attend(None) == Q.QMM_EINVAL
    assert _scored(None) == Q.QMM_EINVAL
    assert _evict(None, n=1) == Q.QMM_EINVAL
    assert _axes(None) == Q.QMM_EINVAL


ATTEND = [
    (dict(q=None), Q.QMM_EINVAL), (dict(O=None), Q.QMM_EINVAL), (dict(T=0), Q.QMM_EINVAL),
    (dict(Hq=0), Q.QMM_EINVAL), (dict(Hq=30), Q.QMM_EINVAL), (dict(N=9), Q.QMM_EINVAL),
    (dict(N=0, cu=PTR), Q.QMM_EINVAL), (dict(scale=float("nan")), Q.QMM_EINVAL),
    (dict(T=257, N=4 * 257), Q.QMM_ESHAPE), (dict(Hq=8 * 65, qs=8 * 65 * 128), Q.QMM_ESHAPE),
    (dict(qs=4095), Q.QMM_ESHAPE), (dict(qs=128), Q.QMM_ESHAPE), (dict(q=PTR + 8), Q.QMM_EALIGN),
    (dict(O=PTR + 4), Q.QMM_EALIGN), (dict(cu=PTR + 3), Q.QMM_EALIGN)]


@pytest.mark.parametrize("kw,code", ATTEND + [
    (dict(null=True), Q.QMM_EINVAL), (dict(table=None), Q.QMM_EINVAL),
    (dict(lens=None), Q.QMM_EINVAL), (dict(first=None), Q.QMM_EINVAL), (dict(G=0), Q.QMM_EINVAL),
    (dict(max_pages=0), Q.QMM_EINVAL), (dict(G=-1), Q.QMM_EINVAL), (dict(G=5), Q.QMM_ESHAPE),
    (dict(max_pages=1 << 27), Q.QMM_ESHAPE), (dict(max_pages=(1 << 27) - 4096, N=1 << 12, cu=PTR), Q.QMM_ESHAPE),
    (dict(N=1 << 27, cu=PTR), Q.QMM_ESHAPE), (dict(par=PTR + 2), Q.QMM_EALIGN),
    (dict(table=PTR + 2), Q.QMM_EALIGN), (dict(lens=PTR + 1), Q.QMM_EALIGN),
    (dict(first=PTR + 2), Q.QMM_EALIGN)])
def test_prefix_refusals(kw, code):
    assert _prefix_attend(_cache(), **kw) == code


@pytest.mark.parametrize("kw,code", ATTEND + [
    (dict(mass=None), Q.QMM_EINVAL), (dict(decay=-0.5), Q.QMM_EINVAL),
    (dict(decay=float("nan")), Q.QMM_EINVAL), (dict(decay=float("inf")), Q.QMM_EINVAL),
    (dict(ms=316), Q.QMM_ESHAPE), (dict(ms=322), Q.QMM_ESHAPE), (dict(ms=-320), Q.QMM_ESHAPE),
    (dict(ms=1 << 38), Q.QMM_ESHAPE), (dict(mass=PTR + 4), Q.QMM_EALIGN)])
def test_scored_refusals(kw, code):
    assert _scored(_cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(mass=None), Q.QMM_EINVAL), (dict(out=None), Q.QMM_EINVAL), (dict(kept=None), Q.QMM_EINVAL),
    (dict(new=None), Q.QMM_EINVAL), (dict(keep=0), Q.QMM_EINVAL), (dict(sinks=-1), Q.QMM_EINVAL),
    (dict(recent=-1), Q.QMM_EINVAL), (dict(sinks=10, recent=7), Q.QMM_EINVAL),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), Q.QMM_EINVAL), (dict(n=0), Q.QMM_EINVAL),
    (dict(n=1025), Q.QMM_EINVAL), (dict(ms=316), Q.QMM_ESHAPE), (dict(ms=322), Q.QMM_ESHAPE),
    (dict(ls=4 * 8 * 320 - 4), Q.QMM_ESHAPE), (dict(ls=4 * 8 * 320 + 2), Q.QMM_ESHAPE),
    (dict(ls=-1 << 20), Q.QMM_ESHAPE), (dict(ls=1 << 48), Q.QMM_ESHAPE),
    (dict(mass=PTR + 8), Q.QMM_EALIGN), (dict(out=(1 << 30) + 4), Q.QMM_EALIGN),
    (dict(kept=(2 << 20) + 2), Q.QMM_EALIGN), (dict(new=(3 << 20) + 1), Q.QMM_EALIGN)])
def test_evict_refusals(kw, code):
    assert _evict([_cache(lens=5 << 20, table=6 << 20)] * 2, **kw) == code


@pytest.mark.parametrize("pools", [
    ((1, 2), (1, 2)), ((1, 2), (1, 3)), ((1, 2), (3, 2)), ((1, 2), (3, 1)), ((1, 1),),
    ((1, 2), (3, 4), (5, 5)), ((1, 2), (3, 4), (5, 6), (7, 8), (6, 9))])
def test_evict_refuses_a_pool_that_stands_twice(pools):
    """Two blocks would move its rows at once."""
    c = [_cache(lens=5 << 20, table=6 << 20, K=k << 34, V=v << 34) for k, v in pools]
    kw = dict(mass=1 << 40, out=1 << 40, ls=4 * 8 * 320)
    assert _evict(c, **kw) == Q.QMM_EINVAL
    for i, x in enumerate(c):
        x.K, x.V = (2 * i + 1) << 34, (2 * i + 2) << 34
    if not torch.cuda.is_available():   # (made-up pointers: never with a device to launch on)
        assert _evict(c, **kw) == Q.QMM_ENODEV


def test_weights_beyond_any_memory_are_refused():
    """B Hkv mass_stride of 2^66 values: no 64-bit sum of them is formed."""
    c = _cache(B=32768, Hkv=32768, lens=5 << 20, table=6 << 20, head_stride=16 * 128,
               page_stride=32768 * 16 * 128, K=1 << 34, V=2 << 34)
    assert _evict([c], mass=1 << 40, out=1 << 40, ls=0, ms=1 << 36) == Q.QMM_ESHAPE
    assert _scored(c, Hq=32768, qs=32768 * 128, N=32768, T=1, ms=1 << 36) == Q.QMM_ESHAPE


# what the call of two layers reads and writes, in 32-bit values
READ = dict(mass=(1 << 28, 2 * 4 * 8 * 320), lens=(2 << 28, 4), table=(3 << 28, 4 * 20))
WRITTEN = dict(out=(4 << 28, 2 * 4 * 8 * 320), kept=(5 << 28, 2 * 4 * 8 * 16), new=(6 << 28, 4))


@pytest.mark.parametrize("out", list(WRITTEN))
@pytest.mark.parametrize("other", list(READ) + list(WRITTEN))
def test_evict_refuses_outputs_over_what_it_reads(out, other):
    if out == other:
        return
    at, n = (READ | WRITTEN)[other]
    # (mass and mass_out are 16-byte aligned; mass_out may be mass itself)
    step = 16 if out == "out" or other in ("out", "mass") else 4
    for place in (at, at + 4 * n - step, at - 4 * WRITTEN[out][1] + step):
        p = {k: v[0] for k, v in (READ | WRITTEN).items()}
        p[out] = place
        if p["out"] == p["mass"]:
            continue
        assert place < at + 4 * n and at < place + 4 * WRITTEN[out][1]
        c = [_cache(lens=p["lens"], table=p["table"], K=(1 + 2 * i) << 34, V=(2 + 2 * i) << 34)
             for i in range(2)]
        assert _evict(c, mass=p["mass"], out=p["out"], kept=p["kept"],
                      new=p["new"]) == Q.QMM_EINVAL


@pytest.mark.parametrize("field", ["table", "lens", "page_stride", "head_stride", "slot_stride",
                                   "B", "num_pages", "page_size", "max_pages", "Hkv", "D", "dtype"])
def test_evict_refuses_caches_that_differ(field):
    other = {"D": 64, "dtype": 1, "page_size": 32}.get(field, getattr(_cache(), field) + 16)
    assert _evict([_cache(), _cache(**{field: other})]) == Q.QMM_EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), Q.QMM_EINVAL), (dict(q=None), Q.QMM_EINVAL), (dict(N=7), Q.QMM_EINVAL),
    (dict(pos=None), Q.QMM_EINVAL), (dict(rope=False), Q.QMM_EINVAL), (dict(axes=False), Q.QMM_EINVAL),
    (dict(dim=0), Q.QMM_EINVAL), (dict(n=0), Q.QMM_EINVAL), (dict(n=9), Q.QMM_EINVAL),
    (dict(n=2), Q.QMM_EINVAL), (dict(axis=[0] * 63 + [3]), Q.QMM_EINVAL),
    (dict(cos_sin=None), Q.QMM_EINVAL), (dict(dim=24), Q.QMM_ESHAPE), (dict(dim=144), Q.QMM_ESHAPE),
    (dict(qs=4100), Q.QMM_ESHAPE), (dict(pos=PTR + 2), Q.QMM_EALIGN), (dict(out=PTR + 8), Q.QMM_EALIGN)])
def test_axes_refusals(kw, code):
    assert _axes(_cache(), **kw) == code


def test_axes_of_pairs_that_are_not_there_are_not_looked_at():
    """The alignment error that ends the call comes behind the checks of the axes."""
    assert _axes(_cache(), dim=16, axis=[0, 1, 2, 0, 1, 2, 0, 1] + [255] * 56,
                 pos=PTR + 2) == Q.QMM_EALIGN


def test_workspaces():
    def prefix(N, **kw):
        return Q.qmm_prefix_attention_workspace_bytes(_cache(**kw), 32, N, 2, 152)

    def scored(T=2, Hq=32, **kw):
        return Q.qmm_scored_attention_workspace_bytes(_cache(**kw), Hq, T, 152)
    assert prefix(8) > 0 and prefix(8) % 16 == 0
    assert prefix(9) - prefix(8) == 2 * 32 * 130 * 4
    assert prefix(8) == prefix(8, max_pages=9000) and prefix(8, B=500) - prefix(8) == 2 * 496 * 8
    assert prefix(0) == 0 and prefix(1 << 27) == 0
    assert scored() > 0 and scored() % 16 == 0
    assert scored(B=8) > scored() and scored(T=257) == 0 and scored(Hq=30) == 0


def test_binding_refuses_what_does_not_fit():
    i = torch.zeros((4, 20), dtype=torch.int32)
    with pytest.raises(TypeError):
        Q.prefix(i, i[:, 0].contiguous(), torch.zeros(5, dtype=torch.int32))
    for bad in ([], [0] * 65, [-1, 0], [8], [0, 1, 9]):
        with pytest.raises(ValueError):
            Q.rope_axes(bad)
    with pytest.raises(ValueError):
        Q.rope_axes([0, 1, 2], axes=2)
    assert Q.rope_axes([0, 1, 1], axes=4).axes == 4 and Q.rope_axes([0, 2]).axes == 3
    rope = Q.qmm_rope(None, None, None, 10, 64, 0, 0.0)
    x = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dim / 2"):
        Q.qmm_kv_append_axes(_cache(), None, x, x, i[:2, :4], Q.rope_axes([0] * 31), rope)
    with pytest.raises(ValueError, match="positions"):
        Q.qmm_kv_append_axes(_cache(), None, x, x, i[:2, :4], Q.rope_axes([0] * 32), rope)


@pytest.mark.parametrize("shape,ok", [((2, 4, 8, 320), True), ((2, 4, 8, 400), True),
                                      ((2, 4, 8, 316), False), ((1, 4, 8, 320), False),
                                      ((2, 8, 4, 320), False), ((4, 8, 320), False)])
def test_binding_shapes_of_the_weights(shape, ok):
    t = torch.zeros(shape)
    if ok:
        assert Q._mass(t, 2, _cache(), "mass") == (32 * shape[3], shape[3])
    else:
        with pytest.raises(ValueError):
            Q._mass(t, 2, _cache(), "mass")


def test_binding_strides_of_the_weights():
    wide = torch.zeros((3, 4, 8, 512))
    assert Q._mass(wide[:2, ..., :320], 2, _cache(), "mass") == (4 * 8 * 512, 512)
    assert Q._mass(wide[1], 1, _cache(), "mass") == (4 * 8 * 512, 512)
    for bad in (wide[:2, ::2], wide[:2, ..., ::2], wide[:2, :, :, :316]):
        with pytest.raises(ValueError):
            Q._mass(bad, 2, _cache(B=bad.shape[1], max_pages=16), "mass") if bad.shape[3] != 316 \
                else Q._mass(bad, 2, _cache(), "mass")
    with pytest.raises(TypeError):
        Q._mass(wide[:2].double(), 2, _cache(), "mass")
