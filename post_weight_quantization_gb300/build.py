"""Build the GPTQ CUDA library (libgptq.so) in-tree for sm_103a, and serving_calls.so beside it.

Each .cu file in csrc/ is compiled by nvcc in parallel, then linked into one shared
library next to this file. The CUDA runtime is linked statically; the only device
code target is sm_103a. serving_calls.so is the Python module of csrc/serving_calls.cpp: host
code that calls the library.

    python -m post_weight_quantization_gb300.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libgptq.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
CALLS_SRC = os.path.join(CSRC, "serving_calls.cpp")
CALLS_PATH = os.path.join(HERE, "serving_calls.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _cxx() -> str:
    return os.environ.get("CXX") or "g++"


def _calls_flags():
    """serving_calls.so is compiled against this torch's C++ headers and says for which: the binding
    does not use it with another."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    return ["-O2", "-std=c++17", "-fPIC", f'-DBUILT_FOR="{torch.__version__}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
            "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")]


def _run(cmd, what: str) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")


def _fingerprint() -> str:
    h = hashlib.sha256()
    files = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h", ".cpp")))
    files.append(os.path.join(INCLUDE, "gptq.h"))
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(ARCH_FLAGS + NVCC_FLAGS + [_cxx(), sys.version] + _calls_flags()).encode())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """Compile and link libgptq.so and serving_calls.so if sources, compilers, torch or Python changed;
    return the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    stamp = os.path.join(BUILD_DIR, "fingerprint")
    fp = _fingerprint()
    if not force and os.path.exists(LIB_PATH) and os.path.exists(CALLS_PATH) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == fp:
                return LIB_PATH
    nvcc = nvcc_path()
    srcs = _sources()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH_FLAGS, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            sys.stderr.write(res.stdout + res.stderr)
        return obj

    calls_obj = os.path.join(BUILD_DIR, "serving_calls.o")
    cxx = _cxx()
    with ThreadPoolExecutor(jobs or min(8, len(srcs) + 1)) as ex:
        calls = ex.submit(_run, [cxx, *_calls_flags(), "-c", CALLS_SRC, "-o", calls_obj], "serving_calls.cpp")
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    calls.result()                               # the library is there even if the module cannot be built
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS_PATH + ".tmp"
    _run([cxx, "-shared", "-o", tmp, calls_obj, "-L", HERE, f"-l:{LIB_NAME}", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
          "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"], "link of serving_calls")
    os.replace(tmp, CALLS_PATH)
    with open(stamp, "w") as f:
        f.write(fp)
    return LIB_PATH


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))


if __name__ == "__main__":
    main()
