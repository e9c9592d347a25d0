"""Build libldn.so (the CUDA library behind include/ldn.h) for sm_103a.

Each .cu file directly under csrc/ is compiled by its own nvcc process (in
parallel), then the objects are linked into lib/libldn.so inside the package.
The diagnostic kernels (csrc/diag/, include/ldn_diag.h) are linked into a
library of their own, lib/libldn_diag.so, which only the tests load.  The native
half of mixer.py (csrc/torch/) is a host-only extension module, lib/_ldn_torch.so,
compiled against the installed torch and linked to libldn.so beside it; without a
torch it is left out, and where it fails libldn.so is in place before that is raised.
The CUDA runtime is linked statically, so the libraries need only the driver at run
time.  Nothing here runs at import time; __graft_entry__.build() and the
tests call build().
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_DIR = os.path.join(HERE, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libldn.so")
DIAG_DIR = os.path.join(CSRC, "diag")
DIAG_LIB_PATH = os.path.join(LIB_DIR, "libldn_diag.so")

TORCH_SRC = os.path.join(CSRC, "torch", "mixer_binding.cpp")
TORCH_LIB_PATH = os.path.join(LIB_DIR, "_ldn_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libldn")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _diag_sources():
    return sorted(os.path.join(DIAG_DIR, f) for f in os.listdir(DIAG_DIR) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return sorted(hs)


def _digest(paths, *words) -> str:
    h = hashlib.sha256()
    for p in paths:
        with open(p, "rb") as f:
            h.update(p.encode() + f.read())
    h.update(" ".join(words).encode())
    return h.hexdigest()


def _stamp() -> str:
    return _digest(_sources() + _diag_sources() + _headers(), *ARCH, *NVCC_FLAGS)


def _torch_stamp():
    """None where there is no torch: the C library is wanted alone."""
    try:
        import torch
    except ImportError:
        return None
    return _digest([TORCH_SRC, os.path.join(INCLUDE, "ldn.h")], torch.__version__)


def _fresh(stamp, name, *libs) -> bool:
    at = os.path.join(OBJ_DIR, name)
    if not all(os.path.exists(p) for p in (*libs, at)):
        return False
    with open(at) as f:
        return f.read() == stamp


def _set_stamp(stamp, name):
    with open(os.path.join(OBJ_DIR, name), "w") as f:
        f.write(stamp)


def _compile(nvcc, src, log_dir):
    tag = "diag_" if os.path.dirname(src) == DIAG_DIR else ""
    obj = os.path.join(OBJ_DIR, tag + os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(log_dir, os.path.basename(src) + ".log"), "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr[-6000:]}")
    return obj


def _compile_torch(log_dir):
    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(OBJ_DIR, "mixer_binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-I", INCLUDE, "-isystem", root, "-isystem",
           os.path.join(root, "torch", "csrc", "api", "include"), "-isystem", cuda, "-isystem",
           sysconfig.get_paths()["include"], "-c", TORCH_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(log_dir, "mixer_binding.cpp.log"), "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {TORCH_SRC}:\n{r.stderr[-6000:]}")
    return obj


def _link_torch(obj):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = TORCH_LIB_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", LIB_DIR, "-l:libldn.so", "-Wl,-rpath,$ORIGIN", "-L", libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _ldn_torch.so failed:\n{r.stderr[-6000:]}")
    os.replace(tmp, TORCH_LIB_PATH)


def _link(nvcc, objs, path):
    tmp = path + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(path)} failed:\n{r.stderr[-6000:]}")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libldn.so and libldn_diag.so, and where torch is installed
    _ldn_torch.so, each if its sources changed; return the path of libldn.so."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    stamp, torch_stamp = _stamp(), _torch_stamp()
    stale = force or not _fresh(stamp, "stamp", LIB_PATH, DIAG_LIB_PATH)
    torch_stale = torch_stamp is not None and (force or not _fresh(torch_stamp, "stamp_torch", TORCH_LIB_PATH))
    if not stale and not torch_stale:
        return LIB_PATH
    srcs, dsrcs = _sources(), _diag_sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, 1 + len(srcs) + len(dsrcs))) as ex:
        torch_obj = ex.submit(_compile_torch, OBJ_DIR) if torch_stale else None
        if stale:
            nvcc = _nvcc()
            objs = list(ex.map(lambda s: _compile(nvcc, s, OBJ_DIR), srcs + dsrcs))
            _link(nvcc, objs[:len(srcs)], LIB_PATH)
            _link(nvcc, objs[len(srcs):], DIAG_LIB_PATH)
            _set_stamp(stamp, "stamp")
    if torch_stale:
        _link_torch(torch_obj.result())
        _set_stamp(torch_stamp, "stamp_torch")
    if verbose:
        for s in srcs + dsrcs:
            with open(os.path.join(OBJ_DIR, os.path.basename(s) + ".log")) as f:
                print(f.read())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
