import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

GOLDEN = os.path.join(ROOT, "tests", "golden")


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")
    config.addinivalue_line("markers", "slow: full-size workload, minutes of host work")
    config.addinivalue_line("markers", "cpu: runs on the host only")


# Cases that hold a value that was wrong, with what is right instead; the tests stay as
# they are, and fail if the wrong value comes back.
SUPERSEDED = {
    "tests/test_gpu_few.py::test_few_refuses[kw0-at most 16]":
        "moe_forward_few takes 1 to 64 tokens, so 17 are not refused: the limit is tested by "
        "test_gpu_few_rows.py::test_few_refuses_past_64_tokens",
}


def pytest_collection_modifyitems(items):
    for item in items:
        if item.nodeid in SUPERSEDED:
            item.add_marker(pytest.mark.xfail(reason=SUPERSEDED[item.nodeid], strict=True))
