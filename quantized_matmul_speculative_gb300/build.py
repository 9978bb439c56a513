"""Build libqmm.so (all CUDA kernels and the C ABI) for sm_103a with nvcc, and
_qmm_torch.so (the native half of the binding for the operators around the product) with g++.

The library needs neither PyTorch nor g++: it is linked first, whatever becomes of
the module, which is left out where PyTorch is not installed and made again for
another version of it or of Python.

Each (bits, group size) instantiation of the tensor-core kernels is its own
translation unit; they compile in parallel.  Objects go to ``_build/`` and the
library lands next to this file.  A rebuild happens only when a source or
header is newer than the library.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD = ROOT / "_build"
LIBRARY = PKG / "libqmm.so"
MODULE = PKG / "_qmm_torch.so"
MODULE_MADE_FOR = BUILD / "qmm_torch.for"  # what module_target() was when the module was linked

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              f"-I{INCLUDE}", f"-I{CSRC}"]

# the C ABI, and the operators around the small-M product
PLAIN_UNITS = ["qmm_api", "qmm_quantize", "qmm_mx_matmul", "qmm_paged", "qmm_verify"]
HEAD_DIMS = [64, 128, 256]
MMA_INSTANCES = [(4, 32), (4, 64), (4, 128), (2, 32), (2, 64), (2, 128), (8, 32), (8, 64), (8, 128)]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not Path(path).exists():
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqmm")
    return path


def units():
    """(source, object, extra flags) for every translation unit."""
    out = [(CSRC / f"{name}.cu", BUILD / f"{name}.o", []) for name in PLAIN_UNITS]
    for d in HEAD_DIMS:
        out.append((CSRC / "qmm_paged_inst.cu", BUILD / f"qmm_paged_d{d}.o", [f"-DQMM_HEAD_DIM={d}"]))
    for bits, gs in MMA_INSTANCES:
        out.append((CSRC / "qmm_mma_inst.cu", BUILD / f"qmm_mma_b{bits}_g{gs}.o",
                    [f"-DQMM_BITS={bits}", f"-DQMM_GS={gs}"]))
    return out


def _inputs():
    files = list(CSRC.glob("*.cu")) + list(CSRC.glob("*.cuh")) + list(CSRC.glob("*.h")) + list(CSRC.glob("*.inc"))
    files += list(CSRC.glob("*.cpp"))
    files += list(INCLUDE.glob("*.h")) + [Path(__file__)]
    return files


def torch_root() -> Path | None:
    """Folder of the installed PyTorch, without importing it; None where there is none."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None or spec.origin is None else Path(spec.origin).resolve().parent


def module_target() -> str:
    """The PyTorch and the Python that a module built now is for; empty without PyTorch."""
    root = torch_root()
    if root is None:
        return ""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return f"{version} {root} {sys.implementation.cache_tag}"


def _newer(target: Path) -> bool:
    return target.exists() and all(f.stat().st_mtime <= target.stat().st_mtime for f in _inputs())


def module_up_to_date() -> bool:
    target = module_target()
    return not target or (_newer(MODULE) and MODULE_MADE_FOR.exists() and MODULE_MADE_FOR.read_text() == target)


def up_to_date() -> bool:
    return _newer(LIBRARY) and module_up_to_date()


def _torch_paths():
    root = torch_root()
    include = [root / "include", root / "include/torch/csrc/api/include", sysconfig.get_paths()["include"],
               Path(nvcc()).resolve().parent.parent / "include", INCLUDE]
    return [f"-I{p}" for p in include], root / "lib"


def _run(cmd, what: str):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stderr}")
    return res.stderr


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> Path:
    BUILD.mkdir(exist_ok=True)
    library, module = force or not _newer(LIBRARY), force or not module_up_to_date()
    jobs = jobs or min(len(units()), os.cpu_count() or 4)
    with ThreadPoolExecutor(max_workers=jobs + 1) as ex:
        module_object = ex.submit(compile_module) if module else None
        if library:
            build_library(ex, verbose)
    if module_object is not None and module_object.result() is not None:  # (raises what the compilation did)
        link_module(module_object.result())
    return LIBRARY


def build_library(ex: ThreadPoolExecutor, verbose: bool = False):
    cc = nvcc()

    def compile_one(unit):
        src, obj, extra = unit
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", str(src), "-o", str(obj)]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        return obj, _run(cmd, f"nvcc for {obj.name}")

    results = list(ex.map(compile_one, units()))
    if verbose:
        for obj, log in results:
            print(f"== {obj.name}\n{log}", file=sys.stderr)
    tmp = LIBRARY.with_name(f"libqmm.{os.getpid()}.tmp.so")
    _run([cc, *ARCH, "-shared", "-o", str(tmp), *[str(o) for o, _ in results]], "link")
    os.replace(tmp, LIBRARY)


def compile_module() -> Path | None:
    """Object of the native half of the binding; None where there is no PyTorch to build it for."""
    if not module_target():
        return None
    flags, _ = _torch_paths()
    obj = BUILD / "qmm_torch.o"
    _run(["g++", "-O2", "-std=c++17", "-fPIC", *flags, "-c", str(CSRC / "qmm_torch.cpp"), "-o", str(obj)],
         f"g++ for {obj.name}")
    return obj


def link_module(obj: Path):
    _, torch_lib = _torch_paths()
    tmp = MODULE.with_name(f"_qmm_torch.{os.getpid()}.tmp.so")
    _run(["g++", "-shared", "-o", str(tmp), str(obj), f"-L{PKG}", "-lqmm", f"-L{torch_lib}", "-ltorch_python",
          "-ltorch_cuda", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"], "module link")
    os.replace(tmp, MODULE)
    MODULE_MADE_FOR.write_text(module_target())


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
