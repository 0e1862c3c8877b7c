import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
HERE = os.path.dirname(os.path.abspath(__file__))
if HERE not in sys.path:
    sys.path.insert(0, HERE)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")
    config.addinivalue_line("markers", "slow: larger CPU oracle cases")


@pytest.fixture(scope="session")
def orc():
    import oracle
    oracle.build()
    return oracle


def pytest_collection_modifyitems(items):
    """test_moe_block_host.py hands stand-in addresses to the library, some of them past its checks, where nothing
    but the missing GPU keeps a kernel from being launched on them: it runs on machines without one only."""
    host = [i for i in items if i.path.name == "test_moe_block_host.py"]
    if host:
        import torch
        if torch.cuda.is_available():
            for i in host:
                i.add_marker(pytest.mark.skip(reason="stand-in addresses: needs a machine without a GPU"))
