"""Build libfp8lm.so (the C-ABI library) in-tree with nvcc for sm_100a, and
_native.so (csrc/binding.cpp, the Python calls of the operators between the GEMMs) with g++.

    python -m fp8_gemms_b200.build [--force] [--verbose]

No fast-math: the cast's scale is one IEEE fp32 division and every product in
the casts and epilogues is a single rounded multiply.
"""
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfp8lm.so")
BINDING = os.path.join(CSRC, "binding.cpp")
NATIVE = os.path.join(PKG, "_native.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]
NATIVE_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                "-Wno-deprecated-declarations"]
NATIVE_LIBS = ["-lfp8lm", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
               "-Wl,-rpath,$ORIGIN"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def _native_key() -> str:
    """What the module is built for and how, beside its sources: it uses PyTorch's C++ headers and
    one Python's.  The places of compiler, CUDA and tree are left out: a built tree can be
    taken to another machine of the same image."""
    import torch
    return "\n".join([torch.__version__, str(torch.version.git_version),
                      str(sysconfig.get_config_var("SOABI")),
                      str(torch._C._GLIBCXX_USE_CXX11_ABI), *NATIVE_FLAGS, *NATIVE_LIBS])


def build_native(force: bool = False) -> str:
    """The Python module beside the library; built for the torch that is installed, which
    NATIVE + ".key" records."""
    deps = [BINDING, os.path.join(INCLUDE, "lm_fp8.h")]
    key, key_file = _native_key(), NATIVE + ".key"
    if not force and os.path.exists(NATIVE) and os.path.exists(key_file):
        with open(key_file) as f:
            same = f.read() == key
        if same and all(os.path.getmtime(p) <= os.path.getmtime(NATIVE) for p in deps):
            return NATIVE
    tmp = NATIVE + ".tmp"
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api",
                                                       "include"),
           os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"),
           sysconfig.get_paths()["include"], INCLUDE]
    subprocess.run([os.environ.get("CXX", "g++"), *NATIVE_FLAGS,
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    *[f"-I{p}" for p in inc], BINDING, "-o", tmp, f"-L{PKG}",
                    "-L" + os.path.join(root, "lib"), *NATIVE_LIBS], check=True)
    os.replace(tmp, NATIVE)
    with open(key_file, "w") as f:
        f.write(key)
    return NATIVE


def build(force: bool = False, verbose: bool = False) -> str:
    build_library(force, verbose)
    build_native(force)
    return LIB


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    objs = []
    for src in sources():
        obj = os.path.join(CSRC, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    subprocess.run([nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp,
                    *objs], check=True)
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
