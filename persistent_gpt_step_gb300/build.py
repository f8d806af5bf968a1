"""Builds libgpt.so in-tree with nvcc for sm_103a (one -gencode, parallel TUs), and
_decode.so, the CPython module through which decode.py hands torch tensors to it (where
torch is installed: the library does not need it).

Usage: python -m persistent_gpt_step_gb300.build [--force]
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgpt.so")
MODULE = os.path.join(HERE, "_decode.so")
SOURCES = ["gpt_host.cu", "kernel_fp32.cu", "kernel_bf16.cu", "kernel_bf16_ext.cu",
           "kv_append.cu", "decode_attention.cu", "decode_bf16_64.cu", "decode_bf16_128.cu", "decode_fp32_64.cu",
           "decode_fp32_128.cu", "next_token.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
         "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgpt.so")


def _deps() -> list[str]:
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    out.append(os.path.join(ROOT, "include", "gpt.h"))
    out.append(os.path.abspath(__file__))
    return out


def _newer_than_sources(path: str) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in _deps())


def _torch() -> str | None:
    """Folder of the installed torch, without importing it."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _built_for() -> str:
    """What _decode.so is compiled against: the Python ABI and the torch that is installed."""
    with open(os.path.join(_torch(), "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{_torch()}\n{f.read()}"


def _stamp() -> str:
    return os.path.join(BUILD, "_decode.built_for")


def _module_up_to_date() -> bool:
    if _torch() is None:
        return True
    if not _newer_than_sources(MODULE) or not os.path.exists(_stamp()):
        return False
    with open(_stamp()) as f:
        return f.read() == _built_for()


def up_to_date() -> bool:
    return _newer_than_sources(LIB) and _module_up_to_date()


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [_nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _module() -> None:
    """Compiles _decode.so (g++) against the installed torch's headers and libraries."""
    torch = _torch()
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = MODULE + ".tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", *["-I" + i for i in inc],
           os.path.join(CSRC, "decode_py.cpp"), "-o", tmp, "-L" + os.path.join(torch, "lib"),
           "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for decode_py.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MODULE)
    with open(_stamp(), "w") as f:
        f.write(_built_for())


def _library(verbose: bool) -> None:
    """Compiles every translation unit and links libgpt.so."""
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(_compile, SOURCES))
    report = "\n".join(r[1] for r in results)
    with open(os.path.join(BUILD, "ptxas.txt"), "w") as f:
        f.write(report)
    if verbose:
        print(report)
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *[r[0] for r in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is missing or out of date (``force``: everything); returns the path of libgpt.so.
    A module that cannot be built is reported after the library has been."""
    library = force or not _newer_than_sources(LIB)
    module = _torch() is not None and (force or not _module_up_to_date())
    if library or module:
        os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(1) as ex:
        made = ex.submit(_module) if module else None
        if library:
            _library(verbose)
        if made:
            made.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
