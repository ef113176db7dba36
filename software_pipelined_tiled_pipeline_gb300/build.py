"""Build libgemmpipe.so (the C-ABI GEMM library) in-tree with nvcc for sm_103a.

Each CUDA translation unit is compiled to an object in parallel under
``_build/`` and the objects are linked into
``software_pipelined_tiled_pipeline_gb300/libgemmpipe.so`` (CUDA runtime linked
statically; the driver is reached through the runtime's entry-point query, so
no libcuda is needed at link time).  Host code is portable C++17: the same
sources build on x86_64 and on aarch64.
"""
import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgemmpipe.so")

SOURCES = ["api.cu", "fp8_api.cu", "k_ffma.cu", "k_fp8_gemm.cu", "k_fp8_norm.cu", "k_fp8_quant.cu", "k_imma.cu",
           "k_umma.cu", "probe.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]

# Kernels whose warps trade registers count on an exact number per thread at launch, and are refused at run time with
# any other: {source: (kernel, registers)}.  ptxas says what it gave them.
LAUNCH_REGISTERS = {"k_fp8_gemm.cu": (r"fp8_ring_kernelILi(128|256)E", 168), "k_umma.cu": (r"umma_i8_overlap_kernel", 128)}


def check_launch_registers(src, ptxas):
    """Raise if a kernel of `src` in ptxas's -v output has other registers than its register split counts on."""
    if src not in LAUNCH_REGISTERS:
        return
    kernel, want = LAUNCH_REGISTERS[src]
    seen = 0
    for part in ptxas.split("Compiling entry function '")[1:]:
        name, used = part.split("'", 1)[0], re.search(r"Used (\d+) registers", part)
        if not re.search(kernel, name):
            continue
        seen += 1
        if used is None or int(used.group(1)) != want:
            raise RuntimeError("%s: %s was compiled to %s registers, its register split counts on %d" % (
                src, name, used.group(1) if used else "an unknown number of", want))
    if not seen:
        raise RuntimeError("%s: no kernel like %s in ptxas's output" % (src, kernel))


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _deps():
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    deps += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    deps.append(os.path.abspath(__file__))
    return deps


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link the library if any source is newer than it; return its path."""
    deps = _deps()
    if not force and not _stale(LIB, deps):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc] + ARCH + CFLAGS + (["-Xptxas", "-v"] if ptxas_verbose or src in LAUNCH_REGISTERS else []) + [
            "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, cmd, r

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    objs = []
    for src, obj, cmd, r in results:
        if verbose or ptxas_verbose:
            print(" ".join(cmd), file=sys.stderr)
            if r.stderr:
                print(r.stderr, file=sys.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        check_launch_registers(src, r.stderr)
        objs.append(obj)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
