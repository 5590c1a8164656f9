"""In-tree build of libfge.so (the C-ABI CUDA library) for sm_103a, and of the Python binding of
its decode-step calls.

Each translation unit under csrc/ is compiled by nvcc in parallel, then linked into
fp8_grouped_expert_gb300/libfge.so; csrc/binding.cpp is compiled by the host compiler against
torch's headers into fp8_grouped_expert_gb300/_decode.so.  A rebuild happens only when a source
or header is newer than the library.  No cmake; plain nvcc, one -gencode.
"""

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfge.so")
BINDING = os.path.join(PKG, "_decode.so")
SOURCES = ["api.cu", "quant.cu", "route.cu", "gemm.cu", "glue.cu", "noalloc.cu", "selftest.cu", "dispatch.cu",
           "decode.cu", "kvcache.cu", "attention.cu", "attention_prefix.cu", "moe_decode.cu"]
HEADERS = ["fge_device.cuh", "chain.cuh", "quotient.cuh", "attention.cuh", "fge_internal.h",
           os.path.join("..", "..", "include", "fge.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I" + os.path.join(ROOT, "include")]


def nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(sources, target):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("command failed: %s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
    return r.stdout + r.stderr


def compile_binding():
    """Compiles csrc/binding.cpp if it changed; returns the object."""
    import torch
    src = os.path.join(CSRC, "binding.cpp")
    obj = os.path.join(BUILD, "binding-torch-%s.o" % torch.__version__)
    header = os.path.join(ROOT, "include", "fge.h")
    if _stale([src, header, __file__], obj):
        home = os.path.join(os.path.dirname(torch.__file__), "include")
        dirs = [home, os.path.join(home, "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"],
                os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
        _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
              "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi()]
             + ["-I" + d for d in dirs] + ["-c", src, "-o", obj])
    return obj


def link_binding(obj):
    """Links the binding from that object if it changed or another torch's is linked."""
    import torch
    record = os.path.join(BUILD, "binding-linked.txt")  # the object that BINDING is from
    linked = None
    if os.path.exists(record):
        with open(record) as f:
            linked = f.read()
    if linked != obj or _stale([obj, LIB], BINDING):
        tmp = BINDING + ".tmp"
        _run(["g++", "-shared", "-o", tmp, obj,
              "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python",
              "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L" + PKG, "-l:libfge.so",
              "-Wl,-rpath,$ORIGIN"])
        if linked is not None:
            os.remove(record)  # whatever happens between here and its rewriting, link again
        os.replace(tmp, BINDING)
        with open(record, "w") as f:
            f.write(obj)


def build(verbose=False, ptxas_info=False):
    """Compile and link libfge.so and the binding if anything changed; returns the library's
    path."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(compile_binding)
        _build_library(verbose, ptxas_info)
        link_binding(binding.result())
    return LIB


def _build_library(verbose, ptxas_info):
    headers = [os.path.join(CSRC, h) for h in HEADERS]
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    if not _stale(srcs + headers + [__file__], LIB) and not ptxas_info:
        return
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        if ptxas_info or _stale([src] + headers + [__file__], obj):
            out = _run([nvcc()] + NVCC_FLAGS + extra + ["-c", src, "-o", obj])
            if verbose or ptxas_info:
                sys.stdout.write(out)
        return obj

    with ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    _run([nvcc()] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv))
