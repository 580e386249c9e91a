"""Build the gfx950 HIP library ``libddpm.so`` in-tree with hipcc, and the binding of
its sequence operators.

    python -m dynamic_dilated_depthwise_amd.build

Every HIP source under ``csrc/`` is compiled to an object in ``_build/`` (in
parallel) and linked into ``dynamic_dilated_depthwise_amd/libddpm.so``.  Packed
fp32 instructions are disabled for all device code.  ``csrc/seq_binding.cpp`` is
host code against torch's headers; it becomes the extension module ``_sequence.so``
beside the library, which it finds there.
"""
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(os.path.dirname(PKG), "_build")
LIB = os.path.join(PKG, "libddpm.so")
BINDING = os.path.join(PKG, "_sequence.so")
ARCH = os.environ.get("DDPM_OFFLOAD_ARCH", "gfx950")

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
CXXFLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-result",
]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *CXXFLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature; drop that line.
    err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{err}")
    if err.strip():
        print(err, file=sys.stderr)
    return obj


def _compile_binding():
    import torch
    from torch.utils.cpp_extension import include_paths
    obj = os.path.join(BUILD, "seq_binding.cpp.o")
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(HIPCC)))
    includes = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(rocm, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-isystem{i}" for i in includes), "-c",
           os.path.join(CSRC, "seq_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for the binding:\n{r.stderr}")
    return obj


def _link_binding(obj):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-shared", obj, "-o", tmp, f"-L{libs}", f"-L{PKG}", "-l:libddpm.so", "-ltorch_python", "-ltorch_cpu",
           "-ltorch_hip", "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)


def build(verbose=True):
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    workers = min(len(srcs), int(os.environ.get("MAX_JOBS", "8")) or 1)
    with ThreadPoolExecutor(max_workers=workers) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    _link_binding(binding.result())
    if verbose:
        print("built", LIB)
        print("built", BINDING)
    return LIB


if __name__ == "__main__":
    build()
