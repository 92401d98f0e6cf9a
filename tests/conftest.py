import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")


# Host tests that pass every argument check with made-up addresses and count on
# the missing device to end the call.  With a GPU the kernel would be launched
# on those addresses, so they run only where there is none.
WITHOUT_GPU_ONLY = {"test_paged.py::test_unused_strides_of_one_row_are_not_checked"}


def pytest_collection_modifyitems(items):
    import torch
    if not torch.cuda.is_available():
        return
    for item in items:
        if os.path.basename(item.nodeid.split("[")[0]) in WITHOUT_GPU_ONLY:
            item.add_marker(pytest.mark.skip(reason="would launch on made-up addresses"))
