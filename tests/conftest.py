import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")


@pytest.fixture(scope="session")
def oracle_lib():
    import oracle
    oracle.build()
    return oracle


# Tests that hold a value that is wrong by what include/qmv.h states.  They stay as they are and run; what they were meant to hold
# is in the test named here.
WRONG = {
    # kv_lens is lowered by the number of queries left out and the queries are expected where they stood before: that is
    # p = kv_lens - max_q + i, where the header has p = kv_lens - n + i with n = q_begin[r + 1] - q_begin[r].  With kv_lens as it
    # was such queries would see tokens behind them.  Held by tests/test_gpu_attention_max_q.py.
    "tests/test_gpu_attention.py::test_rows_of_no_request_and_more_than_max_q":
        "expects query i of n > max_q at kv_lens - max_q + i; it stands at kv_lens - n + i",
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = WRONG.get(item.nodeid.split("[")[0])
        if reason:
            item.add_marker(pytest.mark.xfail(reason=reason, raises=AssertionError, strict=True))
