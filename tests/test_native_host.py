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
            (lambda c: refused(native.state_store_q8, state, c, scales, None, None, 2, 1, 128, None,
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


def test_the_package_works_without_the_compiled_marshalling():
    """Blocked, as on a machine where it was not built: the f32 entries load and check as ever, and a
    low-bit call says what is missing."""
    r = _python("""
import sys
sys.modules["gated_delta_rule_scan_gb300._kda_native"] = None
import torch
from gated_delta_rule_scan_gb300 import kda, mixer
print(kda.abi_version() > 0, kda.library().kda_scan is not None)
try:
    kda.kda_gated_rmsnorm_out(None, None, None, None, rows=1)
except kda.KdaError as e:
    print(e.status)
x, w, s, o = torch.zeros(1, 128), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4), torch.zeros(1, 4)
try:
    kda.kda_proj_w4(x, [w], [s], [o], group=32)
except ImportError as e:
    print("_kda_native.so" in str(e))
""")
    assert r.returncode == 0, r.stderr[-500:]
    assert r.stdout.split() == ["True", "True", "40004", "True"], r.stdout


@pytest.fixture
def scratch_build(tmp_path, monkeypatch):
    """_build with its outputs in a folder of their own and the compilers replaced; the list collects
    what was made."""
    from gated_delta_rule_scan_gb300 import _build
    made = []
    for name, path in (("BUILD_DIR", tmp_path), ("LIB_PATH", tmp_path / "libkda.so"),
                       ("NATIVE_PATH", tmp_path / "_kda_native.so"),
                       ("NATIVE_STAMP", tmp_path / "stamp")):
        monkeypatch.setattr(_build, name, str(path))

    class Done:
        returncode, stderr = 0, ""

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        made.append(os.path.basename(out).split(".tmp")[0])
        open(out, "w").close()
        return Done
    monkeypatch.setattr(_build.subprocess, "run", run)
    return _build, made


def test_a_change_of_torch_rebuilds_the_marshalling(scratch_build, monkeypatch):
    import torch
    build, made = scratch_build
    build.build()
    assert "libkda.so" in made and "_kda_native.so" in made
    made.clear()
    build.build()
    assert made == [] and build.native_matches()
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert not build.native_matches()          # (the package then leaves it unloaded)
    build.build()
    assert made == ["kda_native.cpp.o", "_kda_native.so"]
    made.clear()
    build.build()
    assert made == []


@pytest.mark.parametrize("error", [RuntimeError, FileNotFoundError, ImportError])
def test_without_torchs_headers_the_library_is_built(scratch_build, monkeypatch, error):
    build, made = scratch_build

    def fails():
        raise error("no headers")
    monkeypatch.setattr(build, "_compile_native", fails)
    with pytest.warns(UserWarning, match="no headers"):
        assert build.build() == build.LIB_PATH
    assert "libkda.so" in made and os.path.exists(build.LIB_PATH)
    assert not os.path.exists(build.NATIVE_PATH)


def test_errors_name_the_entry_that_refused(monkeypatch):
    import torch
    from gated_delta_rule_scan_gb300 import kda

    class Refuses:
        def __getattr__(self, name):
            return lambda *args: 40005
    monkeypatch.setattr(kda, "_kda_native", Refuses())
    t = torch.zeros(1)
    for name, call in (
            ("kda_state_store_q8", lambda: kda.kda_state_store_q8(t, t, t, N=1, H=1)),
            ("kda_state_load_q8", lambda: kda.kda_state_load_q8(t, t, t, N=1, H=1)),
            ("kda_decode_fused_q8", lambda: kda.kda_decode_fused_q8(*[t] * 14, N=1, T=1, H=1)),
            ("kda_proj_w4", lambda: kda.kda_proj_w4(t, [t], [t], [t], group=32))):
        assert name in kda.EXPORTED
        with pytest.raises(kda.KdaError, match=name + r"\b") as e:
            call()
        assert e.value.status == 40005
