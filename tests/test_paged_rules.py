"""Paged-cache calls, rules that need no GPU (CPU only)."""
import ctypes
import importlib.util
import os

import pytest
import torch

from split_w4a16_quantized_gb300 import build
from split_w4a16_quantized_gb300 import qmm as Q

PTR = 1 << 20   # an aligned address that no host check follows
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def _cache(**kw):
    c = dict(K=PTR, V=PTR, table=PTR, lens=PTR, page_stride=8 * 16 * 128, head_stride=16 * 128,
             slot_stride=128, B=4, num_pages=100, page_size=16, max_pages=20, Hkv=8, D=128,
             dtype=Q.QMM_CACHE_BF16, k_scale=1.0, v_scale=1.0)
    c.update(kw)
    return Q.qmm_kv_cache(**c)


class _Item:
    def __init__(self, nodeid):
        self.nodeid, self.marks = nodeid, []

    def add_marker(self, mark):
        self.marks.append(mark.name)


@pytest.mark.parametrize("gpu", [False, True])
def test_made_up_addresses_never_reach_a_gpu(gpu, monkeypatch):
    """The host test whose arguments pass every check is left out where a GPU
    would take the launch, and runs where there is none."""
    spec = importlib.util.spec_from_file_location("conftest_rules", os.path.join(HERE, "conftest.py"))
    rules = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(rules)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
    name = "test_unused_strides_of_one_row_are_not_checked"
    items = [_Item("tests/test_paged.py::" + name), _Item("test_paged.py::" + name),
             _Item("tests/test_paged.py::test_null_caches"), _Item("tests/other.py::" + name)]
    rules.pytest_collection_modifyitems(items)
    assert [i.marks for i in items] == ([["skip"], ["skip"], [], []] if gpu else [[]] * 4)


def test_unused_strides_through_the_host_only_entry():
    """A dimension of one row has no stride; over more rows the same strides are
    refused.  The workspace query checks the cache and launches nothing."""
    def nb(**kw):
        return Q.lib().qmm_tree_attention_workspace_bytes(ctypes.byref(_cache(**kw)), kw["Hkv"], 1, 152)
    assert nb(num_pages=1, page_stride=3, Hkv=1, head_stride=-5) > 0
    assert nb(num_pages=2, page_stride=3, Hkv=1, head_stride=-5) == 0
    assert nb(num_pages=1, page_stride=3, Hkv=2, head_stride=-5) == 0
    assert nb(num_pages=1, page_stride=3, Hkv=2, head_stride=16 * 128) > 0


@pytest.mark.parametrize("which", ["q alone", "q_out alone"])
def test_append_takes_q_and_q_out_together(which):
    """Either both or neither, said before anything is asked of the tensors."""
    c = _cache()
    c.device = 0
    x = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q and q_out"):
        Q.qmm_kv_append(c, x if which == "q alone" else None, x, x,
                        None if which == "q alone" else x)
    with pytest.raises(ValueError, match="q and q_out"):
        Q.qmm_kv_append(c, *((x, x, x) if which == "q alone" else (None, x, x, x)))
