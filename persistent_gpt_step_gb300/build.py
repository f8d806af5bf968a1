"""Builds libgpt.so in-tree with nvcc for sm_103a (one -gencode, parallel TUs), and
_decode.so, the CPython module through which decode.py hands torch tensors to it.

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


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MODULE):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(MODULE))
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [_nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _module() -> None:
    """Compiles _decode.so (g++) against the installed torch's headers and libraries."""
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
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


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles every translation unit and links libgpt.so; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        module = ex.submit(_module)
        results = list(ex.map(_compile, SOURCES))
        module.result()
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
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
