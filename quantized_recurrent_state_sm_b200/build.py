"""Build the CUDA library libstepq.so (sm_100a) in-tree with nvcc: one object a
source, compiled side by side, then linked."""
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJECTS = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libstepq.so")
# the checking build (kernels validate the pool's tables before touching
# memory; see stepq_pool_check_guards in include/stepq.h)
LIB_CHECK = os.path.join(HERE, "libstepq_check.so")
SOURCES = ["stepq_abi.cu", "stepq_kernels.cu", "stepq_serve_abi.cu", "stepq_plan.cu", "stepq_prompt.cu",
           "stepq_prompt_tiles.cu", "stepq_prompt_blocks.cu", "stepq_beam.cu"]
HEADERS = ["stepq_internal.cuh", "stepq_device.cuh", "stepq_host.cuh", "stepq_serve.cuh", "stepq_mma.cuh",
           "stepq_tcgen05.cuh", "stepq_prompt_blocks.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    out = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    out.append(os.path.join(ROOT, "include", "stepq.h"))
    return out


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in _deps())


def build(force: bool = False, verbose: bool = False, check: bool = False) -> str:
    """Build libstepq.so, or with check=True the checking build libstepq_check.so
    (-DSTEPQ_CHECK=1)."""
    lib = LIB_CHECK if check else LIB
    if not (force or needs_build(lib)):
        return lib
    flags = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
             "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if check:
        flags.append("-DSTEPQ_CHECK=1")
    if verbose:
        flags.append("-Xptxas=-v")
    objects = []
    jobs = []
    newest = max(os.path.getmtime(os.path.join(CSRC, h)) for h in HEADERS)
    newest = max(newest, os.path.getmtime(os.path.join(ROOT, "include", "stepq.h")))
    os.makedirs(OBJECTS, exist_ok=True)
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(OBJECTS, src[:-3] + ("_check.o" if check else ".o"))
        objects.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) <= max(newest, os.path.getmtime(path)):
            jobs.append([*flags, "-c", path, "-o", obj])
    with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        for f in [ex.submit(subprocess.run, job, check=True) for job in jobs]:
            f.result()
    subprocess.run([nvcc(), *ARCH, "--shared", "-o", lib + ".tmp", *objects], check=True)
    os.replace(lib + ".tmp", lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, check="--check" in sys.argv))
