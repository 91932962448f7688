"""Build libw12.so in-tree: the CUDA kernels for sm_103a (nvcc) plus the host
encoder and the C ABI (g++), linked with the static CUDA runtime so that the
library loads without a GPU driver present (only the calls need one); and,
where torch is installed, kv_host.so, the Python module that takes the paged
cache's calls from torch tensors to the C ABI."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libw12.so")
KV_HOST_PATH = os.path.join(OUT_DIR, "kv_host.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]

CUDA_SOURCES = ["kernels.cu", "kv.cu", "kv_attend_d64.cu", "kv_attend_d128.cu", "kv_attend_d256.cu"]
CXX_SOURCES = ["encoder.cpp", "q8_host.cpp", "capi.cpp"]
KV_HOST_SOURCE = "kv_host.cpp"


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "w12.h"))
    return files


def _torch():
    """torch's directory, without importing it; None where it is not installed."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def _kv_host_made_for():
    """What kv_host.so depends on beside its sources, as text: torch (None: not
    installed, no module to build) and the interpreter."""
    torch = _torch()
    if torch is None:
        return None
    with open(os.path.join(torch, "version.py")) as f:
        return f"{torch}\n{sys.version}\n{f.read()}"


def _stale_file(path) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(f) > os.path.getmtime(path) for f in _inputs())


def _kv_host_stale(made_for) -> bool:
    if made_for is None:
        return False
    if _stale_file(KV_HOST_PATH):
        return True
    try:
        with open(KV_HOST_PATH + ".for") as f:
            return f.read() != made_for
    except OSError:
        return True


def _kv_host_command(out: str):
    # against torch's headers and the libraries that `import torch` has loaded
    torch = _torch()
    libs = os.path.join(torch, "lib")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-Wall", "-I", INCLUDE,
            "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, KV_HOST_SOURCE), "-o", out,
            "-L", libs, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10"]


def build(force: bool = False, verbose: bool = False) -> str:
    made_for = _kv_host_made_for()
    make_lib = force or _stale_file(LIB_PATH)
    make_kv_host = made_for is not None and (force or _kv_host_stale(made_for))
    if not make_lib and not make_kv_host:
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    jobs = []
    objs = []
    for src in CUDA_SOURCES if make_lib else ():
        obj = os.path.join(OUT_DIR, src + ".o")
        cmd = [NVCC, *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xptxas", "-v", "-Xcompiler", "-fPIC",
               "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        jobs.append((cmd, obj))
    for src in CXX_SOURCES if make_lib else ():
        obj = os.path.join(OUT_DIR, src + ".o")
        cmd = [NVCC, "-O3", "-std=c++17", "-Xcompiler", "-fPIC,-Wall,-Wextra,-pthread", "-I", INCLUDE,
               "-x", "cu" if src.endswith(".cu") else "c++", "-c", os.path.join(CSRC, src), "-o", obj]
        jobs.append((cmd, obj))
    kv_host_tmp = KV_HOST_PATH + f".tmp{os.getpid()}"
    if make_kv_host:
        jobs.append((_kv_host_command(kv_host_tmp), None))
    procs = [(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True), cmd, obj)
             for cmd, obj in jobs]
    for p, cmd, obj in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{out}")
        if verbose and out:
            sys.stdout.write(out)
        if obj:
            objs.append(obj)
    if make_kv_host:
        os.replace(kv_host_tmp, KV_HOST_PATH)
        with open(KV_HOST_PATH + ".for", "w") as f:
            f.write(made_for)
    if not make_lib:
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    link = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-pthread", "-cudart", "static"]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(link)}\n{r.stdout}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
