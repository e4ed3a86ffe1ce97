import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# Host tests whose requests pass every check of the host with pointers that are made up: in a
# process that has opened a GPU such a call launches kernels on them.
MADE_UP_POINTERS = {"test_abi_host.py": ("test_requests_at_the_limits_pass_validation",
                                         "test_new_entry_points_valid_requests_pass_validation"),
                    "test_zz_no_alloc.py": ("test_noalloc_size_limit",)}


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long-running full-size check")


def gpu_present():
    import torch
    return torch.cuda.device_count() > 0


def pytest_collection_modifyitems(items):
    named = [i for i in items if i.name in MADE_UP_POINTERS.get(os.path.basename(str(i.fspath)), ())]
    if named and gpu_present():
        for item in named:
            item.add_marker(pytest.mark.skip(reason="a GPU is present: the pointers are not real"))
