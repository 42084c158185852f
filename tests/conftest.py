import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")


def pytest_collection_modifyitems(config, items):
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    if have_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device in this environment")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)


# MEASURED_PEAKS.json holds what a copy and a matrix product reached on the machine at hand, and changes with every
# measurement; the report's expected fractions are those of this one.
REPORT_PEAKS = {"hbm_gbs": 6551.0, "bf16_tflops": 1617.3, "bf16_tflops_sustained": 1379.0}


@pytest.fixture(autouse=True)
def report_peaks(request, monkeypatch):
    if request.module.__name__ == "test_bench_cpu":
        import bench
        monkeypatch.setattr(bench, "load_peaks", lambda: (dict(REPORT_PEAKS), "measured"))
