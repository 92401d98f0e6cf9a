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


PER_DEVICE = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include <atomic>
#include "qmm_per_device.h"
static std::atomic<int> made[100];
static qmm::PerDevice<int> values;
static int value(int device) {   // 0 stands for a device that refused
    return values.get(device, [=] { ++made[device]; return device == 3 ? 0 : 1000 + device; });
}
int main() {
    std::vector<std::thread> threads;
    std::atomic<int> wrong{0};
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&, t] {
            for (int i = 0; i < 500; ++i) {
                const int d = (i * 7 + t) % 66;
                wrong += value(d) != (d == 3 ? 0 : 1000 + d);
            }
        });
    for (auto& t : threads) t.join();
    int once = 0;
    for (int d = 0; d < 64; ++d) once += made[d] == 1;
    std::printf("%d %d %d\n", wrong.load(), once, made[64] > 1 && made[65] > 1);
}
"""


def test_what_belongs_to_a_device_is_asked_once_for_each(tmp_path):
    """The shared-memory opt-in of a kernel and the status word's address: a second
    device gets its own, from whichever thread, and no launch asks twice."""
    import shutil
    import subprocess
    src, exe = tmp_path / "per_device.cpp", tmp_path / "per_device"
    src.write_text(PER_DEVICE)
    csrc = os.path.join(os.path.dirname(HERE), "split_w4a16_quantized_gb300", "csrc")
    subprocess.run([shutil.which("g++"), "-std=c++17", "-O1", "-pthread", "-I", csrc, str(src),
                    "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert out.split() == ["0", "64", "1"]
    for name in ("qmm_tree_attention.cu", "qmm_tree_attention_tc.cu"):
        text = open(os.path.join(csrc, name)).read()
        assert "PerDevice" in text and "once_flag" not in text, name


# tokens, targets, parents, cu, lens, table; path, count, next, new_lens: B = 4,
# T = 2, N = 8, 20 pages a sequence
READ = dict(tokens=(1 << 20, 8), targets=(2 << 20, 8), parents=(3 << 20, 8), cu=(4 << 20, 5),
            lens=(5 << 20, 4), table=(6 << 20, 80))
WRITTEN = dict(path=(7 << 20, 8), count=(8 << 20, 4), next=(9 << 20, 4), new_lens=(10 << 20, 4))


@pytest.mark.parametrize("out", list(WRITTEN))
@pytest.mark.parametrize("other", list(READ) + list(WRITTEN))
def test_accept_refuses_outputs_over_what_it_reads(out, other):
    """Each output against each input and each other output, overlapping by one
    value on either side."""
    if out == other:
        return
    at, n = (READ | WRITTEN)[other]
    for place in (at, at + 4 * (n - 1), at - 4 * (WRITTEN[out][1] - 1)):
        p = {k: v[0] for k, v in (READ | WRITTEN).items()}
        p[out] = place
        arr = (Q.qmm_kv_cache * 1)(_cache(lens=p["lens"], table=p["table"], K=1 << 30, V=2 << 30))
        assert Q.lib().qmm_tree_accept(arr, 1, p["tokens"], p["targets"], p["parents"], p["cu"], 8, 2,
                                       p["path"], p["count"], p["next"], p["new_lens"],
                                       None) == Q.QMM_EINVAL


@pytest.mark.parametrize("scales", [(0.5, 1.0), (1.0, 2.0)])
def test_a_bf16_cache_has_no_scales(scales):
    """Append stores BF16 values as they are, so attention must not scale them."""
    bf16, e4m3 = (_cache(dtype=d, k_scale=scales[0], v_scale=scales[1])
                  for d in (Q.QMM_CACHE_BF16, Q.QMM_CACHE_E4M3))
    nb = Q.lib().qmm_tree_attention_workspace_bytes
    assert nb(ctypes.byref(bf16), 32, 1, 152) == 0 and nb(ctypes.byref(e4m3), 32, 1, 152) > 0
    p = [(20 + i) << 20 for i in range(8)]
    assert Q.lib().qmm_kv_append(ctypes.byref(bf16), None, PTR, PTR, None, 4, 0, 0, 1024, 1024, 0,
                                 None, None, None, None) == Q.QMM_EINVAL
    assert Q.lib().qmm_tree_attention(ctypes.byref(bf16), PTR, 4096, PTR, 4, 1, 32, None, None, 0.0,
                                      PTR, 1 << 30, None) == Q.QMM_EINVAL
    assert Q.lib().qmm_tree_accept((Q.qmm_kv_cache * 1)(bf16), 1, p[0], p[1], None, None, 4, 1, p[2],
                                   p[3], p[4], p[5], None) == Q.QMM_EINVAL
