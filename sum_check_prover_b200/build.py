"""Build libfp.so in-tree with nvcc for sm_100a (cross-compiles without a GPU), and beside it the module _binding, the
layer operators' short way from PyTorch's tensors into it."""

from __future__ import annotations

import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

HERE = Path(__file__).resolve().parent
CSRC = HERE / "csrc"
INCLUDE = HERE.parent / "include"
OBJ = HERE / "_build"
LIB = HERE / "libfp.so"
# (named for the interpreter that it is built for, so that another one does not import it)
BINDING = HERE / ("_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _deps() -> list:
    return sorted(CSRC.glob("*.cuh")) + sorted(CSRC.glob("*.h")) + [INCLUDE / "fp.h"]


def build(force: bool = False, verbose: bool = False, extra: list | None = None) -> Path:
    srcs = sorted(CSRC.glob("*.cu"))
    newest_dep = max(p.stat().st_mtime for p in _deps() + [Path(__file__)])
    OBJ.mkdir(exist_ok=True)
    flags = FLAGS + (extra or [])

    def compile_one(src: Path):
        obj = OBJ / (src.stem + ".o")
        if not force and obj.exists() and obj.stat().st_mtime >= max(src.stat().st_mtime, newest_dep):
            return obj, None
        cmd = [NVCC, *ARCH, *flags, "-c", str(src), "-o", str(obj)]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            return obj, r.stderr + r.stdout
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)
        return obj, None

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        res = list(ex.map(compile_one, srcs))
    errs = [e for _, e in res if e]
    if errs:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errs))
    objs = [o for o, _ in res]
    if force or not LIB.exists() or LIB.stat().st_mtime < max(o.stat().st_mtime for o in objs):
        tmp = LIB.with_suffix(f".so.{os.getpid()}")
        cmd = [NVCC, *ARCH, "-shared", "-o", str(tmp), *map(str, objs)]
        subprocess.run(cmd, check=True, capture_output=not verbose)
        os.replace(tmp, LIB)
    build_binding(force, verbose)
    return LIB


def build_binding(force: bool = False, verbose: bool = False) -> Path | None:
    """Compile csrc/binding.cpp for this interpreter and its PyTorch; None where either lacks what that takes or the
    compiler fails (with a warning: the library is whole, and the operators' methods then do without it)."""
    spec, python = importlib.util.find_spec("torch"), Path(sysconfig.get_paths()["include"])
    root = Path(spec.origin).resolve().parent if spec and spec.origin else None
    if root is None or not all(p.exists() for p in (
            root / "lib" / "libc10_cuda.so", root / "include" / "torch" / "csrc" / "autograd" / "python_variable.h", root / "version.py",
            python / "Python.h")):
        BINDING.unlink(missing_ok=True)
        return None
    (HERE / "_binding.so").unlink(missing_ok=True)  # (an earlier build's name, which every interpreter would import)
    src = CSRC / "binding.cpp"
    newest = max(p.stat().st_mtime for p in (src, INCLUDE / "fp.h", Path(__file__)))
    version = str(runpy.run_path(str(root / "version.py"))["__version__"])
    OBJ.mkdir(exist_ok=True)
    built_for = OBJ / (BINDING.name + ".torch")  # the PyTorch that the module there was compiled against
    if (not force and BINDING.exists() and BINDING.stat().st_mtime >= newest and built_for.exists()
            and built_for.read_text() == version):
        return BINDING
    tmp = BINDING.with_suffix(f".so.{os.getpid()}")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", f'-DFP_TORCH="{version}"', f"-I{root / 'include'}",
           f"-I{python}", f"-I{Path(NVCC).resolve().parents[1] / 'include'}", str(src), "-o", str(tmp),
           f"-L{root / 'lib'}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-L{HERE}", "-l:libfp.so",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = r.stderr + r.stdout if r.returncode else ""
    except OSError as e:
        failed = str(e)
    if failed or not tmp.exists():
        for p in (tmp, BINDING, built_for):  # (an older one may not know the library)
            p.unlink(missing_ok=True)
        warnings.warn(f"{BINDING.name} was not built, the layer operators' calls go without it; {cmd[0]}:\n{failed}")
        return None
    os.replace(tmp, BINDING)
    built_for.write_text(version)
    return BINDING


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
