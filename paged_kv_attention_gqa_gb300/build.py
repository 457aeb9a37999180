"""Build libpkv.so in-tree: nvcc for sm_103a, one process per translation unit; and, where torch is installed, the Python
module _marshal, which hands the tensors of the speculative step's calls to it.

    python -m paged_kv_attention_gqa_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
OUT = os.path.join(PKG, "libpkv.so")
OBJ = os.path.join(PKG, "_build")
SOURCES = ["pkv_api.cu", "decode.cu", "prefill.cu", "prefill_gather.cu", "prefill_pair.cu", "prefill_wide.cu",
           "decode_weights.cu", "weights.cu", "evict.cu", "latent.cu", "latent_dense.cu", "latent_api.cu", "tree.cu", "tree_plan.cu", "tree_api.cu", "maps.cu",
           "planner.cpp", "latent_plan.cpp", "evict_plan.cpp"]
HEADERS = ["plan.h", "launch.h", "handle.h", "latent.h", "evict.h", "tree.h", "decode_kernel.cuh", "ptx.cuh", "tcgen05.cuh", "prefill_kernel.cuh", "prefill_pair.cuh",
           "prefill_wide.cuh"]
MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_folder():
    """Where torch is installed, found without importing it; None where it is not."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec else None


def _torch_mark() -> str:
    """Which torch that is: its place and its version file."""
    folder = _torch_folder()
    try:
        with open(os.path.join(folder, "version.py")) as f:
            return folder + "\n" + f.read()
    except OSError:
        return folder + "\n"


def _marshal_stale() -> bool:
    """The module holds torch's inlined headers and its libraries' place, so it is also stale where torch is another one than
    the one noted beside it."""
    if _stale(MARSHAL, [os.path.join(CSRC, "marshal.cpp"), os.path.join(ROOT, "include", "pkv.h")]):
        return True
    try:
        with open(MARSHAL + ".torch") as f:
            return f.read() != _torch_mark()
    except OSError:
        return True


def _marshal_command(out: str):
    """g++ with torch's headers and libraries."""
    torch = _torch_folder()
    lib = os.path.join(torch, "lib")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-isystem", os.path.join(torch, "include"), "-isystem",
            sysconfig.get_paths()["include"], os.path.join(CSRC, "marshal.cpp"), "-L" + lib, "-ltorch_python", "-ltorch_cpu",
            "-lc10", "-Wl,-rpath," + lib, "-o", out]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(OBJ, exist_ok=True)
    nvcc = _nvcc()
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "pkv.h")]
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"), *extra_flags]
    procs, objs, marshal = [], [], None
    if _torch_folder() is None:  # the library itself is plain C and CUDA
        sys.stderr.write("torch is not installed: _marshal, which the calls of the speculative step need, is not built\n")
    elif force or _marshal_stale():
        marshal = MARSHAL + f".{os.getpid()}.tmp"
        procs.append(("marshal.cpp", subprocess.Popen(_marshal_command(marshal), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(OBJ, src + ".o")
        objs.append(obj)
        if not force and not _stale(obj, [path, *hdrs]):
            continue
        if src.endswith(".cu"):
            cmd = [nvcc, *ARCH, "-lineinfo", *common, "-c", path, "-o", obj]
            if verbose:
                cmd += ["-Xptxas", "-v"]
        else:
            cmd = [nvcc, *common, "-x", "c++", "-c", path, "-o", obj]
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode:
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode:
            failed.append(src)
    if any(src in SOURCES for src in failed):
        raise RuntimeError(f"compilation failed of {failed}")
    if marshal and not failed:
        os.replace(marshal, MARSHAL)
        with open(marshal, "w") as f:
            f.write(_torch_mark())
        os.replace(marshal, MARSHAL + ".torch")
    if force or procs or _stale(OUT, objs):
        tmp = OUT + f".{os.getpid()}.tmp"
        subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt", "-lpthread"],
                       check=True)
        os.replace(tmp, OUT)
    if failed:
        raise RuntimeError(f"compilation failed of {failed} (the library is built)")
    return OUT


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(OUT)
