import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


@pytest.fixture(autouse=True)
def own_draws(request):
    """A GPU test that draws from torch's global generators draws the same in every run, whichever tests ran before it
    (torch seeds them anew for each process)."""
    if request.node.get_closest_marker("gpu"):
        torch.manual_seed(0)
