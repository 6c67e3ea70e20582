"""Builds the HIP library libdgemm.so in-tree for gfx950 with hipcc, and, where torch is installed, the
Python binding of the operators around the product, _binding.so, which calls it.

Each translation unit compiles to an object of its own, all at once (the wide-wave kernels that
read a source matrix sit in gemm_src_*.hip for this; the operators around the product in
ops_*.hip), and the objects are linked into the shared library."""
import importlib.util
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdgemm.so")
SOURCES = [os.path.join(CSRC, name)
           for name in ("gemm.hip", "gemm_src_bf16.hip", "gemm_src_fp8.hip", "ops_block.hip",
                        "ops_block_wide.hip", "ops_quantize.hip", "ops_norm.hip", "ops_clip.hip")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++20", "-fPIC",
    # keep the compiler from forming packed-FP32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


BINDING = os.path.join(CSRC, "binding.cpp")
BINDING_LIB = os.path.join(HERE, "_binding.so")


def binding_command(out):
    """The host compiler (g++, or ROCm's) on the Python binding of the operators, against torch's headers."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cxx = shutil.which("g++") or os.path.join(os.path.dirname(HIPCC), "amdclang++")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f for d in (*include_paths(), sysconfig.get_paths()["include"]) for f in ("-isystem", d)]
    cmd += ["-o", out, BINDING, f"-L{HERE}", "-l:libdgemm.so", "-Wl,-rpath,$ORIGIN"]
    for d in library_paths():
        cmd += [f"-L{d}", f"-Wl,-rpath,{d}"]
    return cmd + ["-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"]


def build_binding(verbose=False):
    cmd = binding_command(BINDING_LIB + ".tmp")
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(BINDING_LIB + ".tmp", BINDING_LIB)

# of one source: the results of its MFMAs go to the registers that vector instructions read
FLAGS_OF = {"ops_block_wide.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def compile_command(src, obj, extra=()):
    return [HIPCC, *FLAGS, *FLAGS_OF.get(os.path.basename(src), ()), *extra, "-c", "-o", obj, src]


def build(verbose: bool = False, extra=()) -> str:
    with tempfile.TemporaryDirectory(prefix="dgemm_build_") as tmp:
        objs = [os.path.join(tmp, os.path.basename(src) + ".o") for src in SOURCES]
        cmds = [compile_command(src, obj, extra) for src, obj in zip(SOURCES, objs)]
        for cmd in cmds:
            if verbose:
                print(" ".join(cmd), flush=True)
        with ThreadPoolExecutor(max_workers=len(cmds)) as pool:
            results = list(pool.map(lambda c: subprocess.run(c), cmds))
        for cmd, res in zip(cmds, results):
            if res.returncode != 0:
                raise subprocess.CalledProcessError(res.returncode, cmd)
        link = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", LIB + ".tmp", *objs]
        if verbose:
            print(" ".join(link), flush=True)
        subprocess.run(link, check=True)
    os.replace(LIB + ".tmp", LIB)
    if importlib.util.find_spec("torch"):
        build_binding(verbose)
    else:   # the C library is whole; only the calls that take torch tensors need the binding
        print("torch is not installed: _binding.so is not built", flush=True)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, extra=[a for a in sys.argv[1:] if a != "-v"]))
