import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")
    config.addinivalue_line("markers", "slow: full-size parity cases (minutes)")


@pytest.fixture(autouse=True)
def argument_structures_stay(request, monkeypatch):
    """test_decode_args hands the library addresses of cache structures that nothing else holds: they live until its end."""
    if request.module.__name__ != "test_decode_args":
        return
    from memory_bound_gemv_gb300 import decode

    made = []

    class Held(decode._KvStruct):
        def __init__(self, *values):
            super().__init__(*values)
            made.append(self)

    monkeypatch.setattr(decode, "_KvStruct", Held)
