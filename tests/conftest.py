import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a GB300 (sm_103a) GPU and the built CUDA library")
    config.addinivalue_line("markers", "slow: full-size parity case (still run by -m gpu)")


@pytest.fixture(autouse=True)
def _same_inputs_every_run():
    """Tests that draw from torch's own generators see the same values in every run and order."""
    import torch
    torch.manual_seed(0)
