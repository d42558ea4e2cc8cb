import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

GOLDEN = os.path.join(ROOT, "tests", "golden")


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Tests that assert what the operator's definition contradicts, left as they are
CONTRADICTED = {
    "test_gpu_adapter.py::test_large_values_in_float16":
        "asserts that every value is infinite where the low-rank value is beyond float16's range; by the definition two "
        "of the 32 are ordinary numbers, y[0][1] = 47735.5 and y[1][5] = -36416.5.  test_gpu_adapter_range.py checks "
        "such values against 64 bits",
}


def pytest_collection_modifyitems(items):
    for item in items:
        for name, reason in CONTRADICTED.items():
            if item.nodeid.endswith(name):
                item.add_marker(pytest.mark.xfail(reason=reason, strict=True))


def load_golden(name):
    with open(os.path.join(GOLDEN, name)) as f:
        return json.load(f)


@pytest.fixture
def golden():
    return load_golden
