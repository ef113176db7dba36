"""Build libgemmpipe.so (the C-ABI GEMM library) in-tree with nvcc for sm_103a.

Each CUDA translation unit is compiled to an object in parallel under
``_build/`` and the objects are linked into
``software_pipelined_tiled_pipeline_gb300/libgemmpipe.so`` (CUDA runtime linked
statically; the driver is reached through the runtime's entry-point query, so
no libcuda is needed at link time).  Beside it ``_torch_ffn.so``, the CPython
extension that takes torch tensors to the feed-forward calls, is compiled with
g++ against the installed torch (without a torch it is left out), once for each
version of torch and Python.  Host code is portable C++17: the same sources
build on x86_64 and on aarch64.
"""
import importlib.metadata
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgemmpipe.so")
TORCH_SOURCE = "torch_ffn.cpp"
TORCH_LIB = os.path.join(PKG, "_torch_ffn.so")
TORCH_STAMP = os.path.join(BUILD, "torch_ffn.for")      # what it was compiled against

SOURCES = ["api.cu", "ffn_api.cu", "fp8_api.cu", "k_ffma.cu", "k_ffn_act.cu", "k_ffn_few.cu", "k_ffn_gated.cu",
           "k_ffn_input_grad.cu", "k_ffn_linear.cu", "k_ffn_weight_grad.cu", "k_fp8_gemm.cu", "k_fp8_norm.cu", "k_fp8_quant.cu", "k_imma.cu", "k_umma.cu", "probe.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]

# Kernels whose warps trade registers count on an exact number per thread at launch, and are refused at run time with
# any other: {source: (kernel, registers)}.  ptxas says what it gave them.
LAUNCH_REGISTERS = {"k_fp8_gemm.cu": (r"fp8_ring_kernelILi(128|256)E", 168),
                    **{"k_ffn_%s.cu" % f: (r"ffn_ring_kernelILi256ELb1ELNS_7RingOutE[123]", 96)
                       for f in ("gated", "input_grad", "linear", "weight_grad")},
                    "k_umma.cu": (r"umma_i8_overlap_kernel", 128)}


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
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".cpp", ".h"))]
    deps += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    deps.append(os.path.abspath(__file__))
    return deps


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch():
    """The torch and the Python that an extension is for, or None where there is no torch."""
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch

        version = torch.__version__
    return "torch %s, %s" % (version, sysconfig.get_config_var("SOABI"))


def _extension_stale(deps) -> bool:
    now = _torch()
    if now is None:
        return False
    try:
        with open(TORCH_STAMP) as f:
            made_for = f.read()
    except OSError:
        made_for = None
    return made_for != now or _stale(TORCH_LIB, deps)


def _build_torch_extension():
    """The CPython extension on torch tensors: host code only, against the torch that is installed."""
    import torch

    base = os.path.dirname(torch.__file__)
    include = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include") if os.path.sep in nvcc() else "/usr/local/cuda/include"]
    tmp = TORCH_LIB + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", os.path.join(CSRC, TORCH_SOURCE), "-o", tmp]
    cmd += ["-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)] + ["-I" + i for i in include]
    lib = os.path.join(base, "lib")
    cmd += ["-L" + lib, "-Wl,-rpath," + lib, "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on %s:\n%s%s" % (TORCH_SOURCE, r.stdout, r.stderr))
    os.replace(tmp, TORCH_LIB)
    with open(TORCH_STAMP, "w") as f:
        f.write(_torch())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link what is older than its sources, the library and the extension; return the library's path."""
    deps = _deps()
    library, extension = force or _stale(LIB, deps), force and _torch() is not None or _extension_stale(deps)
    if not library and not extension:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        beside = ex.submit(_build_torch_extension) if extension else None
        if library:
            _build_library(verbose, ptxas_verbose)
        if beside:
            beside.result()      # (raises once the library is there, which does not need it)
    return LIB


def _build_library(verbose, ptxas_verbose):
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


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
