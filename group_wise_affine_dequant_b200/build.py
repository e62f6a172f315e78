"""Build libnvq.so, the C-ABI library, in-tree for sm_100a, and the Python
extension module _calls that marshals torch tensors into its serving calls.

    python -m group_wise_affine_dequant_b200.build

Each .cu file under csrc/ compiles to an object in _build/ (in parallel), then
nvcc links them into group_wise_affine_dequant_b200/libnvq.so. The CUDA runtime
is linked statically, so the library needs only the NVIDIA driver at run time.
The extension (csrc/torch_calls.cpp, g++ against the installed torch's headers and
Python's) holds no kernels and does not link libnvq.so.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libnvq.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
CALLS = os.path.join(HERE, "_calls.so")


def _calls_sources():
    return CALLS_SRC, os.path.join(INCLUDE, "nvq.h")


def _calls_key() -> str:
    """What the extension depends on: its source, the C interface, torch and Python."""
    import torch

    key = hashlib.sha256(f"{torch.__version__} {sysconfig.get_config_var('SOABI')}".encode())
    for path in _calls_sources():
        with open(path, "rb") as f:
            key.update(f.read())
    return key.hexdigest()


def _key_file() -> str:
    return os.path.join(BUILD, "calls.key")


def calls_current() -> bool:
    """The extension is there and was built from these files against this torch and Python. Where its
    sources are not there, nothing else could be built: then it is taken as it is."""
    if not os.path.exists(CALLS):
        return False
    if not all(os.path.exists(path) for path in _calls_sources()):
        return True
    if not os.path.exists(_key_file()):
        return False
    with open(_key_file()) as f:
        return f.read() == _calls_key()


def build_calls() -> str:
    """Compile the extension module _calls, and note what it was built from."""
    import torch

    home = os.path.dirname(torch.__file__)
    nvcc = shutil.which(NVCC)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc))) if nvcc else "/usr/local/cuda"
    tmp = f"{CALLS}.{os.getpid()}.tmp"  # several processes may build at once
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{home}/include",
           f"-I{home}/include/torch/csrc/api/include", "-I" + sysconfig.get_paths()["include"], f"-I{cuda}/include",
           CALLS_SRC, "-o", tmp, f"-L{home}/lib", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {CALLS_SRC}:\n{r.stderr}")
    os.replace(tmp, CALLS)
    os.makedirs(BUILD, exist_ok=True)
    with open(f"{_key_file()}.{os.getpid()}.tmp", "w") as f:
        f.write(_calls_key())
    os.replace(f.name, _key_file())
    return CALLS


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _sources() + _headers())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _link(objs) -> None:
    tmp = LIB + ".tmp"
    subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)


def build(verbose: bool = False, calls: bool = True) -> str:
    """Build libnvq.so and, with `calls`, the extension. The library is in place whatever becomes of the
    extension, which needs more of the machine (a C++20 compiler, the headers of Python and torch);
    its error is raised behind it."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        extension = ex.submit(build_calls) if calls else None
        _link(list(ex.map(lambda s: _compile(s, verbose), srcs)))
        if extension:
            extension.result()
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
