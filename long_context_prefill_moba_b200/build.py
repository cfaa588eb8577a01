"""Build the MoBA CUDA library (libmoba.so) in-tree for sm_100a, and the torch side of
its serving calls (_moba_torch.so).

    python -m long_context_prefill_moba_b200.build        # or build() from Python
"""
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoba.so")
BINDING = os.path.join(HERE, "_moba_torch.so")
BINDING_SOURCE = os.path.join(CSRC, "torch_binding.cpp")
SOURCES = ["moba_api.cu", "meanpool.cu", "gate.cu", "attn.cu", "attn_f32.cu", "attn_tc.cu", "attn_pair_tc.cu", "attn_bwd.cu", "attn_bwd_tc.cu", "gate_tc.cu", "gate_pooled.cu", "index_check.cu", "norm_rope.cu", "paged_attn.cu", "paged_attn_tc.cu", "paged_decode.cu", "paged_f32.cu", "selftest.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "-Xptxas", "-O3"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    deps.append(os.path.join(ROOT, "include", "moba.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The torch extension over libmoba.so's C calls (host code only)."""
    deps = [BINDING_SOURCE, os.path.join(ROOT, "include", "moba.h")]
    if not force and os.path.exists(BINDING) and all(os.path.getmtime(p) <= os.path.getmtime(BINDING) for p in deps):
        return BINDING
    import torch
    base = os.path.join(os.path.dirname(torch.__file__))
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), sysconfig.get_paths()["include"],
           os.path.join(ROOT, "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-DTORCH_EXTENSION_NAME=_moba_torch",
           *[f"-I{p}" for p in inc], BINDING_SOURCE, "-o", BINDING + ".tmp", "-L", HERE, "-lmoba", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        build_binding(False, verbose)
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [nvcc(), *ARCH, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"], check=True)
    os.replace(tmp, LIB)
    build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
