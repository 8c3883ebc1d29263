import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a GB300 (sm_103a) GPU and the built CUDA library")
    config.addinivalue_line("markers", "slow: large workloads (minutes)")


def pytest_collection_modifyitems(config, items):
    # -m gpu on a machine without a GPU would otherwise error out in fixtures;
    # skip instead so "-m 'not gpu'" and "-m gpu" both behave.
    try:
        import torch
        has_gpu = torch.cuda.is_available()
    except Exception:
        has_gpu = False
    if has_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)


# Written for weights whose scales are powers of two; test_fp8_f32.py runs them with fp32 scales too.
POWERS_OF_TWO = ("test_fp8", "test_moe", "test_mixture")


@pytest.fixture(autouse=True)
def scales_of_weights(request):
    """The scales that the weights of a module's tests have."""
    if request.module.__name__ not in POWERS_OF_TWO:
        yield
        return
    import torch
    from tensor_gemm_reduce_gb300 import fp8
    before = fp8.default_scales()
    fp8.set_default_scales(torch.float8_e8m0fnu)
    yield
    fp8.set_default_scales(before)
