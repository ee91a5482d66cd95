"""Build libdstopk.so in-tree for sm_100a with nvcc (no JIT cache), and next
to it libdstopk_debug.so, the same library compiled with DS_DEBUG (device range
checks that record DS_ERR_RANGE in the status word), and with g++ _front.so, the
Python extension that marshals the usual calls of the 8-bit cache.

    python -m sparse_attention_top_ds_b200.build          # build if stale
    python -m sparse_attention_top_ds_b200.build --force  # always rebuild
"""

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
HEADER = os.path.join(ROOT, "include", "ds_topk.h")
LIB = os.path.join(PKG, "libdstopk.so")
LIB_DEBUG = os.path.join(PKG, "libdstopk_debug.so")
FRONT = os.path.join(PKG, "_front.so")
FRONT_SOURCE = os.path.join(CSRC, "front.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
]


def nvcc_path():
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: cannot build libdstopk.so")


def sources():
    files = [HEADER]
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h")):
            files.append(os.path.join(CSRC, f))
    return files


def stale(lib=LIB):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in sources())


def front_tag():
    """What _front.so is compiled for: this Python and this torch (ImportError without one)."""
    import importlib.metadata
    import sysconfig
    try:
        version = importlib.metadata.version("torch")  # without the seconds that importing it takes
    except importlib.metadata.PackageNotFoundError:
        import torch
        version = torch.__version__
    return f"{sysconfig.get_config_var('SOABI')}, torch {version}"


def front_built_for():
    """The front_tag that _front.so was compiled with, or None."""
    try:
        with open(FRONT + ".tag") as f:
            return f.read()
    except OSError:
        return None


def front_stale():
    if not os.path.exists(FRONT) or front_built_for() != front_tag():
        return True
    t = os.path.getmtime(FRONT)
    return any(os.path.getmtime(f) > t for f in (HEADER, FRONT_SOURCE))


def front_command(out):
    """The g++ command of _front.so: the running Python's headers and its torch's."""
    import sysconfig
    import torch
    gxx = shutil.which("g++")
    if not gxx:
        raise RuntimeError("g++ not found: cannot build _front.so")
    home = os.path.dirname(torch.__file__)
    include = [sysconfig.get_paths()["include"], os.path.join(home, "include"),
               os.path.join(home, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include")]
    return [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            *(f"-I{d}" for d in include), FRONT_SOURCE, "-o", out, "-L" + os.path.join(home, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force=False, verbose=False):
    """Compile csrc/lib.cu into libdstopk.so and libdstopk_debug.so and
    csrc/front.cpp into _front.so next to this file (all side by side); return
    the release library's path.  Without PyTorch the C libraries are all there is to
    build: _front.so serves its tensors only."""
    jobs, errors = [], []
    for lib, extra in ((LIB, []), (LIB_DEBUG, ["-DDS_DEBUG"])):
        if not force and not stale(lib):
            continue
        tmp = lib + ".tmp"
        cmd = [nvcc_path()] + NVCC_FLAGS + extra + ["-o", tmp, os.path.join(CSRC, "lib.cu")]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        proc = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
        jobs.append((lib, tmp, proc))
    tmp = FRONT + ".tmp"
    cmd = None
    try:
        if force or front_stale():
            cmd = front_command(tmp)
    except ImportError as e:
        print(f"_front.so is not built: {e}", file=sys.stderr)
    except (RuntimeError, OSError) as e:
        errors.append(str(e))
    if cmd:
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        jobs.append((FRONT, tmp, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    for lib, tmp, proc in jobs:
        out, err = proc.communicate()
        if proc.returncode != 0:
            errors.append(f"the compiler failed for {os.path.basename(lib)}:\n" + out + err)
        else:
            os.replace(tmp, lib)
            if lib == FRONT:
                with open(FRONT + ".tag", "w") as f:
                    f.write(front_tag())
    if errors:
        raise RuntimeError("\n".join(errors))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
