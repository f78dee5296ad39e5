"""Builds libarx.so (HIP for gfx950) in-tree with hipcc, and _binding.so, the
compiled half of the Python binding, with g++ against torch's headers.

Floating-point flags: no contraction (the sum is adds only, in rank order),
fp32 denormals kept on the GPU, and packed-fp32 instructions disabled. The
host compile pass warns that it does not know the last feature; that is
harmless.
"""
import os
import subprocess
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libarx.so")
SOURCES = [os.path.join(CSRC, f) for f in ("arx_reduce.hip", "arx_sync.hip", "arx_rows.hip", "arx_linear.hip",
                                            "arx_runtime.cpp", "arx_layer.cpp")]
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "arx_binding.cpp")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fno-fast-math", "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def binding_command(out: str) -> list:
    """The g++ line for _binding.so. It sees torch and HIP through their headers
    and libraries alone; the library's functions reach it as addresses."""
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", os.path.join(base, "include"), "-isystem", os.path.join(base, "include/torch/csrc/api/include"),
            "-isystem", sysconfig.get_paths()["include"], "-isystem", "/opt/rocm/include",
            "-I", os.path.join(ROOT, "include"), BINDING_SOURCE, "-o", out,
            "-L" + os.path.join(base, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"]


def build(verbose: bool = False, extra=()) -> str:
    """Compiles the sources side by side, then links."""
    flags = [f for f in FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, os.path.basename(src) + ".o") for src in SOURCES]
        commands = [[HIPCC, *flags, *extra, "-c", src, "-o", obj] for src, obj in zip(SOURCES, objects)]
        link = [HIPCC, "--offload-arch=gfx950", "-shared", *extra, *objects, "-o", LIB + ".tmp", "-lpthread"]
        binding = binding_command(BINDING + ".tmp")
        if verbose:
            for cmd in (*commands, link, binding):
                print(" ".join(cmd), flush=True)
        with ThreadPoolExecutor(4) as pool:
            list(pool.map(lambda cmd: subprocess.run(cmd, check=True), [*commands, binding]))
        subprocess.run(link, check=True)
    os.replace(LIB + ".tmp", LIB)
    os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
