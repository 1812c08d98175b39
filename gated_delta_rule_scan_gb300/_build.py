"""Build libkda.so in-tree with nvcc for sm_103a (GB300), and _kda_native.so, the CPython
marshalling of its latency-bound entry points, with g++ against the installed torch.

One compiler process per translation unit, run in parallel, then one link each.  The library
statically links the CUDA runtime and reaches the driver's tensor-map encoder through the runtime's
entry point query, so it needs no libcuda at link time.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libkda.so")
NATIVE_PATH = os.path.join(PKG, "_kda_native.so")
NATIVE_STAMP = os.path.join(BUILD_DIR, "kda_native.stamp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _cuda_include() -> str:
    """The headers of the toolkit that nvcc belongs to."""
    nvcc = shutil.which(_nvcc()) or "/usr/local/cuda/bin/nvcc"
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")


def _newest_source_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*")) + [os.path.join(ROOT, "include", "kda.h")]
    return max(os.path.getmtime(f) for f in files)


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{' '.join(cmd[:2])} failed:\n{r.stderr}")


def _native_stamp() -> str:
    """What _kda_native.so is bound to besides its source: the interpreter's and torch's ABI."""
    import torch
    return f"{sysconfig.get_config_var('SOABI')} torch {torch.__version__}"


def native_matches() -> bool:
    """Whether _kda_native.so is there and was built for this Python and torch."""
    try:
        with open(NATIVE_STAMP) as f:
            return os.path.exists(NATIVE_PATH) and f.read() == _native_stamp()
    except OSError:
        return False


def _compile_native():
    """kda_native.cpp's object file and torch's library folder."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    obj = os.path.join(BUILD_DIR, "kda_native.cpp.o")
    _run(["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          "-I" + os.path.join(root, "include"),
          "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
          "-I" + sysconfig.get_paths()["include"], "-I" + _cuda_include(),
          "-c", os.path.join(CSRC, "kda_native.cpp"), "-o", obj])
    return obj, os.path.join(root, "lib")


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile every csrc/*.cu for sm_103a and link gated_delta_rule_scan_gb300/libkda.so, and
    csrc/kda_native.cpp into _kda_native.so beside it.  Where the second cannot be built (no torch
    headers, say) the first is there all the same: a warning names the cause, the package works, and
    the calls that need _kda_native.so raise."""
    newest = _newest_source_mtime()
    lib_current = (not force and os.path.exists(LIB_PATH)
                   and os.path.getmtime(LIB_PATH) >= newest)
    native_current = (not force and native_matches()
                      and os.path.getmtime(NATIVE_PATH) >= newest)
    if lib_current and native_current:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    srcs = [] if lib_current else sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        native = None if native_current else ex.submit(_compile_native)
        objs = list(ex.map(compile_one, srcs))
    if not lib_current:
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB_PATH)
    if native is not None:
        try:
            _link_native(*native.result())
        except (ImportError, OSError, RuntimeError) as e:
            # an older one is for other sources or another torch
            for p in (NATIVE_PATH, NATIVE_STAMP):
                if os.path.exists(p):
                    os.remove(p)
            warnings.warn(f"_kda_native.so was not built, the low-bit calls will raise: {e}")
    return LIB_PATH


def _link_native(obj, torch_lib):
    # torch's libraries are loaded before this one; libkda.so is found beside it
    tmp = NATIVE_PATH + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libkda.so", "-L" + torch_lib,
          "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, NATIVE_PATH)
    with open(NATIVE_STAMP, "w") as f:
        f.write(_native_stamp())


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
