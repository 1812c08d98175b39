"""Host-side checks (no GPU) of the compiled marshalling beside libkda.so."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_delta_rule_scan_gb300 import _build
    _build.build()


def _python(code):
    """Runs `code` in a process of its own: what goes wrong here ends the process."""
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                          timeout=300)


# tensors that say they are on a GPU and have no storage, without a GPU
STORAGELESS = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from gated_delta_rule_scan_gb300 import _kda_native as native

def refused(call, *args):
    try:
        call(*args)
    except Exception as e:
        print(type(e).__name__, "storage" in str(e))
    return torch.zeros(1)

with FakeTensorMode():
    def cuda(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    x, w, s, o = cuda(3, 2, 128), cuda(4, 64, dtype=torch.uint8), cuda(4, 4), cuda(2, 4)
    codes, scales, state = cuda(3, 2, 1, 128, 128, dtype=torch.int8), cuda(2, 1, 128), cuda(2, 1, 128, 128)
    for call, t in (
            (lambda x: refused(native.proj_w4, x, [w], [s], None, [o], 32, None, 0), x),
            (lambda c: refused(native.state_move, True, state, c, scales, None, None, 2, 1, 128, None,
                               None, 0), codes),
            (lambda x: refused(native.decode_fused_q8, x, *[x] * 8, codes[0], scales, x, x, x, None, None,
                               None, 2, 1, 1, 1, 128, 4, 0, -5.0, 1e-6, 1.0, 1e-6, 0), x)):
        torch.func.vmap(call)(t)
"""


def test_tensors_without_storage_raise():
    r = _python(STORAGELESS)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert r.stdout.split() == ["RuntimeError", "True"] * 3, r.stdout


def test_streams_come_from_public_calls(monkeypatch):
    """Every entry's default stream is torch.cuda.current_stream's; nothing private stands in."""
    from types import SimpleNamespace
    import torch
    from gated_delta_rule_scan_gb300 import kda

    class OnGpu(torch.Tensor):
        is_cuda, device = True, "cuda:3"
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: SimpleNamespace(cuda_stream=(device, 123)))
    assert kda._stream(None, None, torch.zeros(1).as_subclass(OnGpu)) == ("cuda:3", 123)
    assert kda._stream(5, None) == 5
    assert kda._stream(SimpleNamespace(cuda_stream=7), None) == 7
    assert "torch._C" not in open(kda.__file__).read()
