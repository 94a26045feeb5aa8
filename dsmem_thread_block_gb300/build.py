"""Build libcredit.so in-tree with nvcc for sm_103a.

Each translation unit under csrc/ is compiled in parallel, then linked into
``dsmem_thread_block_gb300/_build/libcredit.so``.  No cmake, one -gencode.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libcredit.so")
# the checked build: the same sources with -DCREDIT_DEBUG (index checks and the
# phase trace), in its own object directory
CHECKED_LIB = os.path.join(BUILD, "libcredit_checked.so")
# the torch layer of the training operators, a Python extension
TORCH_LIB = os.path.join(BUILD, "credit_train_torch.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    p = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(p):
        return p
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libcredit")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    out += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return out


def _stale(lib: str) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in _deps() + [__file__])


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None,
          checked: bool = False) -> str:
    """Compile and link libcredit.so (checked: libcredit_checked.so, with
    -DCREDIT_DEBUG) if any source is newer than it."""
    lib = CHECKED_LIB if checked else LIB
    if not force and not _stale(lib):
        return lib
    objdir = os.path.join(BUILD, "checked") if checked else BUILD
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-Xcompiler", "-Wall", "-I", INCLUDE, "--expt-relaxed-constexpr"]
    if checked:
        flags += ["-DCREDIT_DEBUG"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    flags += list(extra or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        r = subprocess.run([cc, *flags, "-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = lib + f".{os.getpid()}.tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def _torch_root() -> str | None:
    """The directory of the installed torch (None: there is none), without
    importing it."""
    import importlib.util
    try:
        spec = importlib.util.find_spec("torch")
    except ValueError:  # (a module that stands in sys.modules without a spec)
        spec = None
    if spec is None or not spec.submodule_search_locations:
        return None
    return spec.submodule_search_locations[0]


def _torch_stamp(root: str) -> str:
    """What the torch layer is compiled against: the interpreter and the torch."""
    with open(os.path.join(root, "version.py")) as f:
        return f"{sys.version}\n{root}\n{f.read()}"


def build_torch(force: bool = False) -> str:
    """Compile and link the training operators' torch layer
    (csrc/train_torch.cpp) against the installed torch, if out of date: its
    sources, or the torch it was compiled against."""
    import sysconfig
    src = os.path.join(CSRC, "train_torch.cpp")
    deps = [src, os.path.join(INCLUDE, "credit.h"), __file__]
    root = _torch_root()
    if root is None:
        raise RuntimeError("torch not found: its headers are required to build the torch layer")
    stamp, stamp_file, old = _torch_stamp(root), TORCH_LIB + ".stamp", None
    if os.path.exists(stamp_file):
        with open(stamp_file) as f:
            old = f.read()
    if not force and old == stamp and os.path.exists(TORCH_LIB) and \
            os.path.getmtime(TORCH_LIB) >= max(os.path.getmtime(p) for p in deps):
        return TORCH_LIB
    os.makedirs(BUILD, exist_ok=True)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    tmp = TORCH_LIB + f".{os.getpid()}.tmp"
    r = subprocess.run(
        [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE,
         "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
         "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
         "-isystem", cuda, src, "-o", tmp, "-L", os.path.join(root, "lib"), "-ltorch_python",
         "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(stamp_file):
        os.remove(stamp_file)  # none stands beside a library it does not describe
    os.replace(tmp, TORCH_LIB)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return TORCH_LIB


def build_all(force: bool = False) -> tuple[str, str]:
    """Both libraries and, where torch is installed, the torch layer, compiled
    side by side: (regular, checked).  The libraries need no torch; a torch
    layer that does not compile raises after both are there."""
    with cf.ThreadPoolExecutor(max_workers=3) as ex:
        reg = ex.submit(build, force)
        chk = ex.submit(build, force, False, None, True)
        layer = ex.submit(build_torch, force) if _torch_root() else None
        libs = reg.result(), chk.result()
        if layer:
            layer.result()
        return libs


if __name__ == "__main__":
    if "--checked" in sys.argv:
        print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, checked=True))
    else:
        print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
