"""Builds libhpcdecode.so (nvcc, sm_103a only) and the binding's extension module
_tensors.so (g++, against the installed PyTorch) in the package directory.

The library's translation units are compiled in parallel and linked with the
CUDA runtime statically, so it needs nothing at run time beyond the NVIDIA
driver.  Each is rebuilt only when a source or header is newer, the module also
for another PyTorch or Python.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import tempfile
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB_PATH = os.path.join(HERE, "libhpcdecode.so")
EXT_PATH = os.path.join(HERE, "_tensors.so")
EXT_SOURCE = os.path.join(CSRC, "tensors.cpp")
EXT_STAMP = EXT_PATH + ".stamp"  # what the module was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libhpcdecode.so")


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(f) > t for f in _inputs())


def extension_target() -> str:
    """What _tensors.so depends on beside its source: it looks into PyTorch's own
    structures, so a module of another PyTorch or Python is not one to load."""
    import torch
    return f"{torch.__version__} {torch.__file__} {sysconfig.get_config_var('SOABI')} " \
           f"abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def extension_built_for() -> str | None:
    """extension_target() of the module in the tree ("" if it does not say), None without one."""
    if not os.path.exists(EXT_PATH):
        return None
    try:
        with open(EXT_STAMP) as f:
            return f.read()
    except FileNotFoundError:
        return ""


def build_extension(force: bool = False) -> str:
    """Compile _tensors.so, the check of a call's tensors."""
    target = extension_target()
    if not force and extension_built_for() == target and \
            os.path.getmtime(EXT_PATH) > max(os.path.getmtime(f) for f in (EXT_SOURCE, __file__)):
        return EXT_PATH
    import torch
    base = os.path.dirname(torch.__file__)
    staged = EXT_PATH + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(base, "include"),
           "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"), EXT_SOURCE,
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-o", staged]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {EXT_SOURCE}:\n{res.stderr}")
    os.replace(staged, EXT_PATH)
    with open(staged, "w") as f:
        f.write(target)
    os.replace(staged, EXT_STAMP)
    return EXT_PATH


def build(force: bool = False, verbose: bool = False, defines=(), out: str | None = None) -> str:
    """Compile the library (to `out`, default the package's libhpcdecode.so) and, beside the
    package's own, the binding's extension module.  That needs g++ and PyTorch's headers, which
    a caller of the C ABI need not have: where it cannot be made the library is, with a
    warning (build_extension() raises, and so do the calls that need the module).

    `defines` are extra -D settings, e.g. the pipeline shape of the attention
    kernels (HPC_BF16_STAGES, HPC_BF16_TPS, HPC_FP8_STAGES, HPC_FP8_TPS)."""
    target = out or LIB_PATH
    own = out is None and not defines
    with ThreadPoolExecutor(1) as pool:  # beside the library's compilation
        extension = pool.submit(build_extension, force) if own else None
        if force or not own or is_stale():
            _build_library(target, verbose, defines)
        if extension:
            try:
                extension.result()
            except (RuntimeError, OSError, ImportError) as e:
                warnings.warn(f"the binding's extension module _tensors was not built: {e}")
    return target


def _build_library(target: str, verbose: bool, defines) -> None:
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                    "--expt-relaxed-constexpr"] + [f"-D{d}" for d in defines]
    with tempfile.TemporaryDirectory(prefix="hpcdecode_build_") as tmp:
        def compile_one(src):
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            cmd = [nvcc, *flags, "-c", src, "-o", obj]
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
            if verbose and res.stderr:
                print(res.stderr)
            return obj

        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            objs = list(pool.map(compile_one, sources()))
        out_tmp = os.path.join(tmp, "libhpcdecode.so")
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", out_tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr}")
        staged = target + f".{os.getpid()}.tmp"
        shutil.copyfile(out_tmp, staged)
        os.replace(staged, target)


if __name__ == "__main__":
    import argparse
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--define", "-D", action="append", default=[])
    ap.add_argument("--out", default=None)
    a = ap.parse_args()
    print(build(force=True, verbose=True, defines=a.define, out=a.out))
