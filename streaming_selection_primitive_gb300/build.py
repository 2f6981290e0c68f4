"""Builds libprofk.so (the C-ABI library) in-tree for sm_103a.

Each translation unit is compiled by nvcc in parallel, then linked with
``nvcc -shared`` (CUDA runtime linked statically, so the library only needs the
driver at run time).  Objects go to ``_build/``; the library to ``lib/``.
A unit is recompiled when it or any header is newer than its object.  The
language-model selections' Python half (csrc/binding.cpp) is compiled by g++
against the installed torch and linked to the library, which needs neither: it
is linked first, and without torch it is all that is built.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
CSRC = PKG / "csrc"
INCLUDE = PKG.parent / "include"
BUILD = PKG / "_build"
LIBDIR = PKG / "lib"
LIB = LIBDIR / "libprofk.so"
BINDING_SOURCE = CSRC / "binding.cpp"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", str(INCLUDE)] + ARCH
SOURCES = ["sample.cu", "select.cu", "sort.cu", "refine.cu", "tie.cu", "rows.cu", "filter.cu", "segments.cu", "api.cu", "params.cpp", "noalloc.cu", "tokens.cu", "route.cu", "route_scores.cu",
           "api_lm.cu", "logprobs.cu", "head.cu", "api_logprobs.cu"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or Path(cand).exists()):
            return cand
    return "nvcc"


def _headers_mtime() -> float:
    hs = list(CSRC.glob("*.h")) + list(CSRC.glob("*.cuh")) + list(INCLUDE.glob("*.h"))
    return max((h.stat().st_mtime for h in hs), default=0.0)


def _compile(src: Path, obj: Path, verbose: bool) -> None:
    cmd = [_nvcc()] + NVCC_FLAGS + ["-c", str(src), "-o", str(obj)]
    if src.suffix == ".cpp":
        cmd = [_nvcc(), "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", str(INCLUDE), "-c", str(src), "-o", str(obj)]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src.name}:\n{r.stdout}\n{r.stderr}")


def binding_path() -> Path:
    """The native half of _lm.py, for the torch that is installed (its C++ interface differs by version)."""
    import torch
    return LIBDIR / f"profk_torch-{torch.__version__}.so"


def _compile_binding(obj: Path, verbose: bool) -> None:
    import sysconfig

    import torch
    home = Path(torch.__file__).resolve().parent
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for inc in (home / "include", home / "include" / "torch" / "csrc" / "api" / "include",
                sysconfig.get_paths()["include"], Path(_nvcc()).resolve().parent.parent / "include"):
        cmd += ["-isystem", str(inc)]
    _run(cmd + ["-c", str(BINDING_SOURCE), "-o", str(obj)], BINDING_SOURCE.name, verbose)


def _link_binding(obj: Path, out: Path, verbose: bool) -> None:
    import torch
    home = Path(torch.__file__).resolve().parent / "lib"
    tmp = out.with_suffix(".so.tmp")
    _run(["g++", "-shared", "-o", str(tmp), str(obj), f"-L{LIBDIR}", "-l:libprofk.so", "-Wl,-rpath,$ORIGIN", f"-L{home}",
          f"-Wl,-rpath,{home}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"],
         "the binding", verbose)
    os.replace(tmp, out)


def _run(cmd, what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building {what} failed:\n{r.stdout}\n{r.stderr}")


def _binding_jobs(force: bool):
    """(object, library, whether the object is stale) of the binding; None without torch."""
    try:
        out = binding_path()
    except ModuleNotFoundError:
        return None
    obj = BUILD / (out.stem + ".o")
    stale = force or not obj.exists() or obj.stat().st_mtime < max(BINDING_SOURCE.stat().st_mtime, _headers_mtime())
    return obj, out, stale


def build(verbose: bool = False, force: bool = False) -> Path:
    """Compiles what is stale and links lib/libprofk.so; returns its path.  A
    binding that does not compile raises after that."""
    BUILD.mkdir(exist_ok=True)
    LIBDIR.mkdir(exist_ok=True)
    hdr = _headers_mtime()
    binding = _binding_jobs(force)
    jobs = []
    for name in SOURCES:
        src = CSRC / name
        obj = BUILD / (name + ".o")
        if force or not obj.exists() or obj.stat().st_mtime < max(src.stat().st_mtime, hdr):
            jobs.append((src, obj))
    with ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
        # (Among the library's units, not to be waited for by itself.)
        extra = ex.submit(_compile_binding, binding[0], verbose) if binding and binding[2] else None
        list(ex.map(lambda j: _compile(j[0], j[1], verbose), jobs))
        objs = [BUILD / (n + ".o") for n in SOURCES]
        newest = max(o.stat().st_mtime for o in objs)
        if force or jobs or not LIB.exists() or LIB.stat().st_mtime < newest:
            tmp = LIB.with_suffix(".so.tmp")
            cmd = [_nvcc(), "-shared"] + ARCH + ["-o", str(tmp)] + [str(o) for o in objs]
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB)
        if extra is not None:
            extra.result()
    if binding is None:
        if verbose:
            print("no torch: the library alone", flush=True)
        return LIB
    obj, out, _ = binding
    if force or not out.exists() or out.stat().st_mtime < obj.stat().st_mtime:
        _link_binding(obj, out, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
