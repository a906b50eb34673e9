"""Build libbi.so (the CUDA kernels and the C ABI of include/bi.h) for sm_100a with nvcc.

The library is built in-tree next to the Python binding, with the CUDA runtime
linked statically, so it loads without a GPU and carries no JIT cache.
"""
import os
import subprocess
import sys

CSRC = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(CSRC)
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
SOURCES = [os.path.join(CSRC, "bi.cu")]
DEPS = SOURCES + [os.path.join(CSRC, n) for n in ("gemm.cuh", "gemm_pair.cuh", "rowops.cuh", "maxsum.cuh", "ptx.cuh", "attention.cuh",
                                                  "rope.cuh", "paged_attention.cuh", "token_logprobs.cuh")] + [
    os.path.join(INCLUDE, "bi.h")]
LIB = os.path.join(PKG, "libbi.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared", "-cudart", "static",
]


def nvcc():
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def build(force: bool = False, out: str = LIB, defines=(), verbose: bool = False) -> str:
    if not force and os.path.exists(out):
        newest = max(os.path.getmtime(p) for p in DEPS)
        if os.path.getmtime(out) >= newest:
            return out
    cmd = [nvcc(), *NVCC_FLAGS, "-I" + INCLUDE, *[f"-D{d}" for d in defines]]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    cmd += ["-o", out, *SOURCES, "-ldl", "-lpthread", "-lrt"]
    subprocess.run(cmd, check=True)
    return out


MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")


def marshal_current() -> bool:
    """Whether the extension module is there, newer than its sources and built against this torch."""
    import torch
    deps = [MARSHAL_SRC, os.path.join(INCLUDE, "bi.h")]
    if not os.path.exists(MARSHAL) or os.path.getmtime(MARSHAL) < max(os.path.getmtime(p) for p in deps):
        return False
    with open(MARSHAL, "rb") as f:
        return f"built for torch {torch.__version__};".encode() in f.read()


def build_marshal(force: bool = False) -> str:
    """The binding's extension module (argument marshalling only; no kernels), against torch's headers."""
    if not force and marshal_current():
        return MARSHAL
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", f'-DBI_TORCH_VERSION="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + INCLUDE, "-I" + os.path.join(root, "include"),
           "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"), "-o", MARSHAL, MARSHAL_SRC,
           "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    subprocess.run(cmd, check=True)
    return MARSHAL


PROBE_SRC = os.path.join(CSRC, "mma_probe.cu")
PROBE = os.path.join(PKG, "mma_probe")


def build_probe(force: bool = False) -> str:
    """The tcgen05 MMA cost probe (a stand-alone program, not part of libbi.so)."""
    deps = [PROBE_SRC, os.path.join(CSRC, "ptx.cuh")]
    if not force and os.path.exists(PROBE) and os.path.getmtime(PROBE) >= max(os.path.getmtime(p) for p in deps):
        return PROBE
    cmd = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-I" + CSRC, "-o", PROBE,
           PROBE_SRC]
    subprocess.run(cmd, check=True)
    return PROBE


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    print(build_marshal(force="--force" in sys.argv))
