"""Build libdgc.so for gfx950 with hipcc, and, where torch and g++ are there,
the torch module over it, in-tree.

    python -m sparsified_gradient_compression_amd.build

Floating-point flags: no FMA contraction, IEEE denormals kept, and packed
FP32 instructions disabled, so every binary32 operation rounds once, as the
method's arithmetic is defined.
"""

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libdgc.so")
BINDING = os.path.join(LIBDIR, "_dgc_torch.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
SOURCES = [os.path.join(CSRC, f) for f in
           ("dgc_api.hip", "dgc_gradset.hip", "dgc_layers.hip", "layers_bf16.hip", "layers_fp16.hip")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in
                     ("launch_grid.hpp", "layers.hpp", "layers_big.hpp", "layers_direct.hpp", "layers_elem.hpp", "layers_guarded.hpp", "layers_mid.hpp", "layers_thin.hpp", "layers_launch.hpp", "layers_tile.hpp",
                      "dgc_device.hpp", "kernel_fused.hpp", "kernels_binlocal.hpp", "kernels_sampled.hpp",
                      "kernels_compress.hpp", "kernels_codec.hpp", "kernels_shared.hpp", "kernels_tensor.hpp")] + [os.path.join(ROOT, "include", "dgc.h")]

ARCH = os.environ.get("DGC_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-ffp-contract=off",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-I", os.path.join(ROOT, "include"),
    "-I", CSRC,
]


def binding_command(out):
    """g++ on the torch module: no GPU code, torch's headers and C++ ABI, and libdgc.so beside it."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    include = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], "/opt/rocm/include",
                                               os.path.join(ROOT, "include")]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
            + [f for i in include for f in ("-isystem", i)]
            + [BINDING_SOURCE, "-o", out, "-L", LIBDIR, "-l:libdgc.so", "-Wl,-rpath,$ORIGIN",
               "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"])


def hipcc():
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    return exe


def has_binding():
    """Whether the torch module can be built here.  The library itself needs hipcc alone."""
    return importlib.util.find_spec("torch") is not None and shutil.which("g++") is not None


def build(verbose=True):
    """Compile libdgc.so and the torch module over it (always recompiles)."""
    os.makedirs(LIBDIR, exist_ok=True)
    tmp = LIB + ".tmp"
    compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)

    objects = [os.path.join(LIBDIR, os.path.basename(s) + ".o") for s in SOURCES]
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as pool:
        list(pool.map(lambda so: run([hipcc()] + compile_flags + ["-c", so[0], "-o", so[1]]),
                      zip(SOURCES, objects)))
    run([hipcc(), f"--offload-arch={ARCH}", "-shared"] + objects + ["-o", tmp])
    os.replace(tmp, LIB)
    for o in objects:
        os.remove(o)
    if has_binding():
        run(binding_command(BINDING + ".tmp"))
        os.replace(BINDING + ".tmp", BINDING)
    elif os.path.exists(BINDING):
        os.remove(BINDING)  # of another library
    return LIB


def is_stale():
    built, sources = [LIB], list(DEPENDS)
    if has_binding():
        built.append(BINDING)
        sources.append(BINDING_SOURCE)
    if not all(map(os.path.exists, built)):
        return True
    t = min(map(os.path.getmtime, built))
    return any(os.path.getmtime(f) > t for f in sources)


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
