"""Paged-cache calls, host side (CPU only): argument errors come back as codes
before any CUDA work, workspace sizes, and the binding's own checks."""
import ctypes

import pytest
import torch

from split_w4a16_quantized_gb300 import build
from split_w4a16_quantized_gb300 import qmm as Q

PTR = 1 << 20   # an aligned address that no host check follows


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def _cache(**kw):
    c = dict(K=PTR, V=PTR, table=PTR, lens=PTR, page_stride=8 * 16 * 128, head_stride=16 * 128,
             slot_stride=128, B=4, num_pages=100, page_size=16, max_pages=20, Hkv=8, D=128,
             dtype=Q.QMM_CACHE_BF16, k_scale=1.0, v_scale=1.0)
    c.update(kw)
    return Q.qmm_kv_cache(**c)


BAD_CACHES = [
    (dict(K=None), Q.QMM_EINVAL), (dict(V=None), Q.QMM_EINVAL), (dict(table=None), Q.QMM_EINVAL),
    (dict(lens=None), Q.QMM_EINVAL), (dict(B=0), Q.QMM_EINVAL), (dict(num_pages=0), Q.QMM_EINVAL),
    (dict(page_size=0), Q.QMM_EINVAL), (dict(max_pages=0), Q.QMM_EINVAL),
    (dict(Hkv=0), Q.QMM_EINVAL), (dict(dtype=2), Q.QMM_EINVAL), (dict(dtype=-1), Q.QMM_EINVAL),
    (dict(k_scale=0.0), Q.QMM_EINVAL), (dict(v_scale=-1.0), Q.QMM_EINVAL),
    (dict(k_scale=float("nan")), Q.QMM_EINVAL), (dict(v_scale=float("inf")), Q.QMM_EINVAL),
    (dict(D=96), Q.QMM_ESHAPE), (dict(D=256), Q.QMM_ESHAPE), (dict(page_size=4), Q.QMM_ESHAPE),
    (dict(page_size=24), Q.QMM_ESHAPE), (dict(page_size=131072), Q.QMM_ESHAPE),
    (dict(max_pages=1 << 28), Q.QMM_ESHAPE), (dict(B=70000), Q.QMM_ESHAPE),
    (dict(slot_stride=0), Q.QMM_ESHAPE), (dict(slot_stride=130), Q.QMM_ESHAPE),
    (dict(head_stride=64), Q.QMM_ESHAPE), (dict(page_stride=-128), Q.QMM_ESHAPE),
    (dict(page_stride=1 << 40), Q.QMM_ESHAPE), (dict(slot_stride=136, dtype=1), Q.QMM_ESHAPE),
    (dict(K=PTR + 8), Q.QMM_EALIGN), (dict(V=PTR + 2), Q.QMM_EALIGN),
    (dict(table=PTR + 2), Q.QMM_EALIGN), (dict(lens=PTR + 1), Q.QMM_EALIGN),
]


def _append(cache, q=PTR, k=PTR, v=PTR, out=PTR, N=8, Hq=32, qs=4096, ks=1024, vs=1024, os=4096,
            cu=None, pos=None, rope=None):
    return Q.lib().qmm_kv_append(ctypes.byref(cache) if cache is not None else None, q, k, v, out,
                                 N, Hq, qs, ks, vs, os, cu, pos,
                                 ctypes.byref(rope) if rope is not None else None, None)


def _attend(cache, q=PTR, qs=4096, O=PTR, N=8, T=2, Hq=32, cu=None, par=None, scale=0.0, ws=PTR,
            nb=1 << 30):
    return Q.lib().qmm_tree_attention(ctypes.byref(cache) if cache is not None else None, q, qs, O,
                                      N, T, Hq, cu, par, scale, ws, nb, None)


def _accept(caches, tok=PTR, tgt=PTR, par=PTR, cu=None, N=8, T=2, path=PTR, count=PTR, nxt=PTR,
            new=PTR + 64, n=None):
    arr = (Q.qmm_kv_cache * max(1, len(caches)))(*caches) if caches is not None else None
    return Q.lib().qmm_tree_accept(arr, n if n is not None else len(caches), tok, tgt, par, cu, N,
                                   T, path, count, nxt, new, None)


@pytest.mark.parametrize("bad,code", BAD_CACHES, ids=[str(b[0]) for b in BAD_CACHES])
def test_bad_caches_refused_by_every_call(bad, code):
    c = _cache(**bad)
    assert _append(c, cu=PTR) == code
    assert _attend(c, cu=PTR) == code
    assert _accept([_cache(), c] if code == Q.QMM_EINVAL else [c, c], cu=PTR) == code
    assert Q.lib().qmm_tree_attention_workspace_bytes(ctypes.byref(c), 32, 2, 152) == 0


def test_unused_strides_of_one_row_are_not_checked():
    c = _cache(num_pages=1, page_stride=3, Hkv=1, head_stride=-5)
    # every host check passes: what is left is the missing device
    assert _append(c, Hq=1, qs=128, ks=128, vs=128, os=128) == Q.QMM_ENODEV or \
        torch.cuda.is_available()


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), Q.QMM_EINVAL), (dict(v=None), Q.QMM_EINVAL), (dict(q=None), Q.QMM_EINVAL),
    (dict(out=None), Q.QMM_EINVAL), (dict(Hq=0), Q.QMM_EINVAL), (dict(Hq=-1), Q.QMM_EINVAL),
    (dict(N=0), Q.QMM_EINVAL), (dict(N=7), Q.QMM_EINVAL), (dict(N=-4), Q.QMM_EINVAL),
    (dict(qs=4100), Q.QMM_ESHAPE), (dict(qs=2048), Q.QMM_ESHAPE), (dict(ks=1020), Q.QMM_ESHAPE),
    (dict(vs=0), Q.QMM_ESHAPE), (dict(os=8), Q.QMM_ESHAPE), (dict(os=4104), Q.QMM_ESHAPE),
    (dict(q=PTR + 2), Q.QMM_EALIGN), (dict(k=PTR + 8), Q.QMM_EALIGN),
    (dict(v=PTR + 4), Q.QMM_EALIGN), (dict(out=PTR + 8), Q.QMM_EALIGN),
    (dict(cu=PTR + 2), Q.QMM_EALIGN), (dict(pos=PTR + 1), Q.QMM_EALIGN)])
def test_append_refusals(kw, code):
    assert _append(_cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dim=-16), Q.QMM_EINVAL), (dict(cos_sin=None), Q.QMM_EINVAL), (dict(rows=0), Q.QMM_EINVAL),
    (dict(interleaved=2), Q.QMM_EINVAL), (dict(q_norm=PTR, eps=-1.0), Q.QMM_EINVAL),
    (dict(k_norm=PTR, eps=float("nan")), Q.QMM_EINVAL), (dict(dim=24), Q.QMM_ESHAPE),
    (dict(dim=144), Q.QMM_ESHAPE), (dict(cos_sin=PTR + 4), Q.QMM_EALIGN),
    (dict(q_norm=PTR + 2), Q.QMM_EALIGN), (dict(k_norm=PTR + 8), Q.QMM_EALIGN)])
def test_rope_refusals(kw, code):
    r = dict(cos_sin=PTR, rows=100, dim=128, interleaved=0, eps=1e-6)
    r.update(kw)
    assert _append(_cache(), rope=Q.qmm_rope(**r)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), Q.QMM_EINVAL), (dict(O=None), Q.QMM_EINVAL), (dict(T=0), Q.QMM_EINVAL),
    (dict(Hq=0), Q.QMM_EINVAL), (dict(Hq=30), Q.QMM_EINVAL), (dict(N=9), Q.QMM_EINVAL),
    (dict(N=0, cu=PTR), Q.QMM_EINVAL), (dict(scale=float("nan")), Q.QMM_EINVAL),
    (dict(T=257, N=4 * 257), Q.QMM_ESHAPE), (dict(Hq=8 * 65, qs=8 * 65 * 128), Q.QMM_ESHAPE),
    (dict(qs=4095), Q.QMM_ESHAPE), (dict(qs=128), Q.QMM_ESHAPE), (dict(q=PTR + 8), Q.QMM_EALIGN),
    (dict(O=PTR + 4), Q.QMM_EALIGN), (dict(par=PTR + 2), Q.QMM_EALIGN),
    (dict(cu=PTR + 3), Q.QMM_EALIGN)])
def test_attention_refusals(kw, code):
    assert _attend(_cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(tok=None), Q.QMM_EINVAL), (dict(tgt=None), Q.QMM_EINVAL), (dict(path=None), Q.QMM_EINVAL),
    (dict(count=None), Q.QMM_EINVAL), (dict(T=0), Q.QMM_EINVAL), (dict(N=9), Q.QMM_EINVAL),
    (dict(new=PTR), Q.QMM_EINVAL), (dict(n=0), Q.QMM_EINVAL), (dict(n=1025), Q.QMM_EINVAL),
    (dict(T=257, N=4 * 257), Q.QMM_ESHAPE), (dict(tok=PTR + 2), Q.QMM_EALIGN),
    (dict(path=PTR + 1), Q.QMM_EALIGN), (dict(nxt=PTR + 2), Q.QMM_EALIGN),
    (dict(new=PTR + 66), Q.QMM_EALIGN)])
def test_accept_refusals(kw, code):
    assert _accept([_cache()] * 2, **kw) == code


@pytest.mark.parametrize("field", ["table", "lens", "page_stride", "head_stride", "slot_stride",
                                   "B", "num_pages", "page_size", "max_pages", "Hkv", "D", "dtype"])
def test_accept_refuses_caches_that_differ(field):
    other = {"D": 64, "dtype": 1, "page_size": 32}.get(field, getattr(_cache(), field) + 16)
    assert _accept([_cache(), _cache(**{field: other})], new=PTR + 256) == Q.QMM_EINVAL


def test_null_caches():
    assert _append(None) == Q.QMM_EINVAL
    assert _attend(None) == Q.QMM_EINVAL
    assert _accept(None, n=1) == Q.QMM_EINVAL
    assert Q.lib().qmm_tree_attention_workspace_bytes(None, 32, 2, 152) == 0


def test_workspace_does_not_grow_with_batch_or_length():
    a = Q.qmm_tree_attention_workspace_bytes(_cache(), 32, 8, 152)
    assert a > 0 and a % 16 == 0
    assert a == Q.qmm_tree_attention_workspace_bytes(_cache(B=512, max_pages=9000), 32, 8, 152)
    assert Q.qmm_tree_attention_workspace_bytes(_cache(), 32, 257, 152) == 0
    assert Q.qmm_tree_attention_workspace_bytes(_cache(), 30, 8, 152) == 0


def test_binding_refuses_host_tensors():
    t = torch.zeros((4, 8, 16, 128), dtype=torch.bfloat16)
    i = torch.zeros((4, 20), dtype=torch.int32)
    with pytest.raises(TypeError):
        Q.kv_cache(t, t, i, i[:, 0].contiguous())
    with pytest.raises(TypeError):
        Q.rope(torch.zeros((10, 128)))
