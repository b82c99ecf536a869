"""Builds libsvt.so from csrc/ with nvcc for sm_103a (one -gencode, translation units
compiled in parallel, static CUDA runtime), and beside it _binding.so, the Python binding of its
short calls (g++, against the installed torch's headers). Both land next to this file."""

from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
LIB = PKG / "libsvt.so"
BINDING = PKG / "_binding.so"
BINDING_SOURCE = CSRC / "binding.cpp"
BUILD_DIR = PKG / "_build"
# The phase-trace build: the same sources with SVT_PHASE_TRACE defined (clock stamps at each
# pipeline step of the attention kernel); a separate library that only profiling loads.
TRACE_LIB = PKG / "libsvt_trace.so"
TRACE_BUILD_DIR = PKG / "_build_trace"
SOURCES = ["api.cu", "attention.cu", "resolve.cu", "union.cu", "merge.cu", "noalloc.cu", "topk.cu", "probe.cu",
           "pair_prefill.cu", "rope.cu", "distill.cu", "backward.cu", "api_layer.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-lineinfo",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def binding_target() -> str:
    """What a binding is good for: the Python and the torch whose headers it was compiled against."""
    import torch

    return f"Python {sys.version_info.major}.{sys.version_info.minor}, torch {torch.__version__}"


def _binding_command(out: Path) -> list:
    import torch

    root = Path(torch.__file__).resolve().parent
    cuda = Path(_nvcc()).resolve().parent.parent if os.path.sep in _nvcc() else Path("/usr/local/cuda")
    include = [root / "include", root / "include/torch/csrc/api/include", sysconfig.get_paths()["include"],
               cuda / "include", INCLUDE]
    libs = ["torch_python", "torch", "torch_cpu", "torch_cuda", "c10", "c10_cuda"]
    return ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", str(BINDING_SOURCE), "-o", str(out),
            f'-DSVT_BINDING_TARGET="{binding_target()}"',
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-isystem{i}" for i in include),
            f"-L{root / 'lib'}", f"-Wl,-rpath,{root / 'lib'}", *(f"-l{name}" for name in libs)]


def binding_up_to_date() -> bool:
    # (its text holds the target's name, so that no other Python or torch has to load it to find out)
    if not BINDING.exists() or binding_target().encode() + b"\0" not in BINDING.read_bytes():
        return False
    t = BINDING.stat().st_mtime
    return all(p.stat().st_mtime <= t for p in (BINDING_SOURCE, INCLUDE / "svt.h", Path(__file__)))


def _inputs():
    return [CSRC / s for s in SOURCES] + list(CSRC.glob("*.cuh")) + list(CSRC.glob("*.h")) + [INCLUDE / "svt.h"]


def up_to_date(lib: Path = LIB) -> bool:
    if not lib.exists():
        return False
    t = lib.stat().st_mtime
    return all(p.stat().st_mtime <= t for p in _inputs())


def build(force: bool = False, verbose: bool = False, trace: bool = False) -> Path:
    """Builds libsvt.so (or, with trace=True, the phase-trace library) and the binding, and returns the
    library's path."""
    lib = TRACE_LIB if trace else LIB
    build_dir = TRACE_BUILD_DIR if trace else BUILD_DIR
    flags = NVCC_FLAGS + (["-DSVT_PHASE_TRACE"] if trace else [])
    binding = None
    if force or not binding_up_to_date():
        binding_tmp = BINDING.with_suffix(f".so.tmp{os.getpid()}")
        binding = subprocess.Popen(_binding_command(binding_tmp), stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                   text=True)
    if force or not up_to_date(lib):
        _build_library(lib, build_dir, flags, verbose)
    if binding is not None:
        out, _ = binding.communicate()
        if binding.returncode != 0:
            raise RuntimeError("g++ failed:\n--- binding.cpp\n" + out)
        os.replace(binding_tmp, BINDING)
    return lib


def _build_library(lib: Path, build_dir: Path, flags: list, verbose: bool) -> None:
    build_dir.mkdir(exist_ok=True)
    nvcc = _nvcc()
    procs = []
    objs = []
    for src in SOURCES:
        obj = build_dir / (Path(src).stem + ".o")
        objs.append(obj)
        cmd = [nvcc, *flags, "-c", str(CSRC / src), "-o", str(obj)]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        if pr.returncode != 0:
            failed.append(f"--- {src}\n{out}")
        elif verbose and out.strip():
            print(out)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
    tmp = lib.with_suffix(f".so.tmp{os.getpid()}")
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-o", str(tmp), *map(str, objs)]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout)
    os.replace(tmp, lib)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
