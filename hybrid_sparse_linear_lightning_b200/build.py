"""Build libsala.so in-tree with nvcc for sm_100a (no GPU needed to compile)."""
from __future__ import annotations

import json
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from importlib.metadata import version

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libsala.so")
CALLS = os.path.join(PKG, "_packed.so")           # Python module of the packed-batch calls, on libsala.so
REPORT = os.path.join(PKG, "libsala.ptxas.json")
CALLS_SOURCE = os.path.join(CSRC, "packed_calls.cpp")
SOURCES = ["api.cu", "packed.cu"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]
LINK_FLAGS = [
    "-shared",
    # the decoder block's GEMMs
    "-lcublasLt", "-Xlinker", "-rpath,/usr/local/cuda/lib64",
]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def built_for() -> dict:
    """What the Python module depends on besides its sources: another one of these needs another build."""
    return {"torch": version("torch"), "python": sysconfig.get_config_var("SOABI")}


def needs_build() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(CALLS) and os.path.exists(REPORT)):
        return True
    with open(REPORT) as f:
        if json.load(f).get("built_for") != built_for():
            return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "sala.h")]
    return any(os.path.getmtime(p) > t for p in deps if os.path.isfile(p))


# Kernels whose in-kernel register reallocation (setmaxnreg) is sized for a
# fixed launch allocation: the build fails unless ptxas gave each exactly
# this many registers per thread, so a library that built cannot hang on a
# register split larger than its launch allocation.
REGISTER_SPLIT_KERNELS = {"linear_segout_kernel": 128}
PACKED_SPLIT_KERNELS = {"dense_attn_kernel": 168, "prefix_attn_kernel": 168,
                        "linear_packed_kernel": 128}


def parse_ptxas(text: str) -> dict:
    """{mangled kernel name: registers per thread} from `ptxas -v` output."""
    regs, cur = {}, None
    for line in text.splitlines():
        m = re.search(r"Compiling entry function '([^']+)'", line)
        if m:
            cur = m.group(1)
            continue
        m = re.search(r"Used (\d+) registers", line)
        if m and cur:
            regs[cur] = int(m.group(1))
            cur = None
    return regs


def check_register_splits(regs: dict, splits: dict = REGISTER_SPLIT_KERNELS) -> None:
    for short, want in splits.items():
        got = {k: v for k, v in regs.items() if short in k}
        if not got:
            raise RuntimeError(f"ptxas report has no entry for {short}")
        bad = {k: v for k, v in got.items() if v != want}
        if bad:
            raise RuntimeError(f"{short}: built with {sorted(set(bad.values()))} registers per "
                               f"thread; its register split needs exactly {want}")


def calls_command(out: str) -> list:
    """Compile and link the Python module against torch's headers and libraries."""
    import torch
    at = os.path.dirname(torch.__file__)
    inc = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")]
    lib = os.path.join(at, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *["-isystem" + i for i in inc],
            "-o", out, CALLS_SOURCE, LIB + ".tmp", "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not needs_build():
        return LIB
    obj_dir = os.path.join(PKG, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    objs = [os.path.join(obj_dir, s + ".o") for s in SOURCES]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise subprocess.CalledProcessError(r.returncode, cmd)
        return r.stdout + r.stderr

    def compile_one(src_obj):
        src, obj = src_obj
        return run([nvcc_path(), *NVCC_FLAGS, "-Xptxas", "-v", *extra, "-I",
                    os.path.join(ROOT, "include"), "-c", "-o", obj, os.path.join(CSRC, src)])

    with ThreadPoolExecutor(len(SOURCES)) as pool:   # one nvcc per source, side by side
        text = "".join(pool.map(compile_one, zip(SOURCES, objs)))
    run([nvcc_path(), *NVCC_FLAGS, *LINK_FLAGS, "-Xlinker", "-soname,libsala.so", "-o", LIB + ".tmp", *objs])
    run(calls_command(CALLS + ".tmp"))
    cur = ""
    for line in text.splitlines():
        m = re.search(r"Function properties for (\S+)", line)
        if m:
            cur = m.group(1)
        if re.search(r"[1-9]\d* bytes spill", line) or "warning" in line.lower():
            sys.stderr.write(f"{cur}: {line.strip()}\n")
    regs = parse_ptxas(text)
    check_register_splits(regs)
    check_register_splits(regs, PACKED_SPLIT_KERNELS)
    with open(REPORT, "w") as f:
        json.dump({"registers_per_thread": regs, "built_for": built_for()}, f, indent=1, sort_keys=True)
    os.replace(LIB + ".tmp", LIB)
    os.replace(CALLS + ".tmp", CALLS)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
