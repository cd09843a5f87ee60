import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
GOLDEN = os.path.join(ROOT, "tests", "golden")


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Cases whose expected values contradict the definition they test.  They run, and are expected to fail.
WRONG_VALUES = {
    # In pages of 48, say, row 1 keeps 20 tokens of a sequence of which row 13 keeps 83: the reference
    # leaves row 1 the page of block 0 to write to, because it had one holder before the call, while row 13
    # reads its every token.  test_fork_of_shared_pools has the same inputs with the definition's values.
    "test_gpu_tree.py::test_fork[300-8-6-48-20-9-any-True]": "two rows of the result write and read one page",
    "test_gpu_tree.py::test_fork[9000-40-300-16-70-310-any-True]": "two rows of the result write and read one page",
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = WRONG_VALUES.get(item.nodeid.split("/")[-1])
        if reason:
            item.add_marker(pytest.mark.xfail(reason=reason, strict=True, raises=AssertionError))


@pytest.fixture(scope="session")
def golden_dir():
    return GOLDEN
