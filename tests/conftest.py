import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

GOLDEN = os.path.join(ROOT, "tests", "golden")


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: long-running CPU test")


# Host tests that make accepted calls with addresses of no memory: without a GPU such a call ends with the
# library's CUDA error; on one it would launch a kernel that reads them.
NO_MEMORY = ("test_abi.py", "test_attention_abi.py", "test_attention_limits.py")


def reaches_no_gpu(items, cuda_available):
    """The tests of a session that may run, with every GPU hidden where none of them needs one; where there
    is a GPU and tests that need it, those of NO_MEMORY that do not are left for a session of their own."""
    if not any(item.get_closest_marker("gpu") for item in items):
        os.environ["CUDA_VISIBLE_DEVICES"] = ""
        return list(items)
    if not cuda_available():
        return list(items)
    return [item for item in items
            if item.get_closest_marker("gpu") or os.path.basename(str(item.path)) not in NO_MEMORY]


@pytest.hookimpl(trylast=True)   # (after -m and -k have chosen; CUDA reads the variable when it is first used)
def pytest_collection_modifyitems(config, items):
    def cuda_available():
        import torch

        return torch.cuda.is_available()

    keep = reaches_no_gpu(items, cuda_available)
    if len(keep) < len(items):
        kept = set(keep)
        config.hook.pytest_deselected(items=[item for item in items if item not in kept])
        items[:] = keep


def golden_lines(name):
    """Non-comment, non-empty lines of a fixture under tests/golden/."""
    with open(os.path.join(GOLDEN, name)) as f:
        for line in f:
            line = line.strip()
            if line and not line.startswith("#"):
                yield line


@pytest.fixture(scope="session")
def orc():
    import oracle

    oracle.lib()
    return oracle
