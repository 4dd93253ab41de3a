import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")
    config.addinivalue_line("markers", "slow: long CPU oracle runs")


# Tests whose expected value was shown to be wrong: each still runs as it was
# written, and has to fail.  {(file, test): what is wrong with its value}
_WRONG_VALUES = {
    ("test_gpu_int8.py", "test_layer_with_a_large_y"):
        "expects the layer's y rounded to bf16 before the aggregation: that adds up to "
        "sum |w y| 2^-8 to an output, which is to be within one rounding of the exact sum "
        "(test_gpu_int8_layer.py holds it to that)",
}


def pytest_collection_modifyitems(items):
    for item in items:
        why = _WRONG_VALUES.get((item.path.name, getattr(item, "originalname", None)))
        if why:
            item.add_marker(pytest.mark.xfail(reason=why, strict=True, raises=AssertionError))


@pytest.fixture(scope="session")
def oracle_lib():
    import oracle

    oracle._load()
    return oracle
