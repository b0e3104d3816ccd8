import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")


@pytest.fixture(scope="session")
def oracle():
    from oracle import oracle as O
    O.build(force=False)
    return O


# Its model counts, at one step, tokens of a request that kv_reserve refused and that
# no call ever stored (773 tokens in 7 blocks of 128, a run of 129, no free block, step
# 33: it wants 807).  test_gpu_pages_refused.py holds histories to the definition.
COUNTS_REFUSED = "tests/test_gpu_pages.py::test_histories[1-128]"


def pytest_collection_modifyitems(items):
    for item in items:
        if item.nodeid.endswith(COUNTS_REFUSED):
            item.add_marker(pytest.mark.xfail(strict=True, reason="its model counts tokens of a refused request"))
