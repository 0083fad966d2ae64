"""Build libfp4gemv.so from csrc/ with nvcc for sm_103a (GB300).

Each translation unit compiles in its own nvcc process (in parallel); the
objects are linked into ``moe_nvfp4_gemv_gb300/libfp4gemv.so`` against the
shared CUDA runtime.  csrc/marshal.cpp becomes ``_marshal.so`` beside it, an
extension module on this interpreter's torch (g++, at the same time).  Rebuilds
only when a source or header is newer than what it makes, and the extension
module also for another interpreter or torch than it was built for.  Usage:
``python -m moe_nvfp4_gemv_gb300.build [--force]``.
"""
from __future__ import annotations

import glob
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfp4gemv.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_FOR = os.path.join(BUILD_DIR, "marshal_for.txt")  # what it was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libfp4gemv needs the CUDA toolkit to build")


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.inc")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def _marshal_for() -> str:
    """What the extension module depends on besides its sources: its binary interfaces, and where torch's are."""
    import torch
    return "\n".join((torch.__version__, _torch_dir(), str(torch.compiled_with_cxx11_abi()), sys.version,
                      platform.machine()))


def _marshal_stale() -> bool:
    if not os.path.exists(MARSHAL) or not os.path.exists(MARSHAL_FOR):
        return True
    with open(MARSHAL_FOR) as f:
        if f.read() != _marshal_for():
            return True
    t = os.path.getmtime(MARSHAL)
    deps = [os.path.join(CSRC, "marshal.cpp"), os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _start_marshal(nvcc: str) -> tuple[str, subprocess.Popen]:
    """Starts the compiler of _marshal.so; the path it writes to, and the process."""
    import torch
    tdir, cuda = _torch_dir(), os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", INCLUDE, "-isystem", os.path.join(tdir, "include"),
           "-isystem", os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
           os.path.join(CSRC, "marshal.cpp"), "-o", tmp, "-L", os.path.join(tdir, "lib"), "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + os.path.join(tdir, "lib")]
    return tmp, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish_marshal(tmp: str, proc: subprocess.Popen) -> None:
    out, _ = proc.communicate()
    if proc.returncode != 0:
        sys.stderr.write(out.decode(errors="replace"))
        raise RuntimeError("the C++ compiler failed for marshal.cpp")
    os.makedirs(BUILD_DIR, exist_ok=True)
    if os.path.exists(MARSHAL_FOR):
        os.remove(MARSHAL_FOR)
    os.replace(tmp, MARSHAL)
    with open(MARSHAL_FOR, "w") as f:
        f.write(_marshal_for())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of libfp4gemv.so."""
    library, marshal = force or _stale(), force or _marshal_stale()
    if not library and not marshal:
        return LIB
    nvcc = _nvcc()
    started = _start_marshal(nvcc) if marshal else None
    try:
        if library:
            _build_library(nvcc, verbose)
    finally:
        if started:
            _finish_marshal(*started)
    return LIB


def _build_library(nvcc: str, verbose: bool) -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    if verbose:
        common += ["-Xptxas", "-v"]
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        procs.append((src, subprocess.Popen([nvcc, *common, "-c", src, "-o", obj],
                                            stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        if verbose or pr.returncode != 0:
            sys.stderr.write(out.decode(errors="replace"))
        if pr.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(os.path.basename(f) for f in failed))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "shared",
                           "-Xlinker", "-rpath," + _cuda_lib_dir(nvcc)])
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
