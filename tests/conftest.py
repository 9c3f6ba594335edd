import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

# Tests without the gpu mark call the library with made-up device addresses, also in calls whose arguments are valid:
# on a machine with a GPU they would launch kernels on unmapped memory. So GPUs are hidden while tests are collected,
# and shown again only to a run of gpu tests alone (-m gpu); in any other run those are skipped.
HIDDEN = "KDA_TESTS_HIDDEN_DEVICES"  # what was visible, for the worker processes of a parallel run


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: long-running CPU test")
    if not hasattr(config, "workerinput"):
        os.environ[HIDDEN] = os.environ.get("CUDA_VISIBLE_DEVICES", "all")
    os.environ["CUDA_VISIBLE_DEVICES"] = ""


@pytest.hookimpl(trylast=True)  # after tests are deselected by mark and name
def pytest_collection_modifyitems(items):
    if all(item.get_closest_marker("gpu") for item in items):
        visible = os.environ.get(HIDDEN, "all")
        if visible == "all":
            os.environ.pop("CUDA_VISIBLE_DEVICES", None)
        else:
            os.environ["CUDA_VISIBLE_DEVICES"] = visible
        return
    for item in items:
        if item.get_closest_marker("gpu"):
            item.add_marker(pytest.mark.skip(reason="the GPU is hidden from a run with other tests: run with -m gpu"))
