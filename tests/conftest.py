import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

GOLDEN = os.path.join(ROOT, "tests", "golden")


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: full-size shapes (seconds of oracle work)")


def golden_lines(name):
    """Non-comment, non-empty lines of a fixture, with trailing '#' comments removed."""
    out = []
    with open(os.path.join(GOLDEN, name)) as f:
        for line in f:
            line = line.split("#", 1)[0].strip()
            if line:
                out.append(line.split())
    return out


@pytest.fixture(scope="session")
def orc():
    import oracle
    oracle.lib()
    return oracle


@pytest.fixture(autouse=True)
def fills_before_calls(request, monkeypatch):
    """test_gpu_logprobs.call fills the outputs and the workspace on the current stream; a call on another stream has to
    wait for that, or it runs beside the fills and may find its workspace overwritten."""
    module = request.module
    if module.__name__ != "test_gpu_logprobs":
        return
    made = module.call

    class Waiting:
        def __init__(self, pn, torch):
            self.pn, self.torch = pn, torch

        def __getattr__(self, name):
            return getattr(self.pn, name)

        def logprobs(self, *args, stream=None, **kw):
            if stream is not None:
                stream.wait_stream(self.torch.cuda.current_stream())
            return self.pn.logprobs(*args, stream=stream, **kw)
    monkeypatch.setattr(module, "call", lambda pn, torch, *a, **kw: made(Waiting(pn, torch), torch, *a, **kw))
