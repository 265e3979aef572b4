"""Builds the CUDA library in-tree: ``exact_io_aware_68_b200/libfa_sm100.so`` for sm_100a.

    python -m exact_io_aware_68_b200.build [-v]

The whole library is one translation unit (``csrc/fa_api.cu`` includes the kernels); the CUDA
runtime is linked statically and the driver's tensor-map encoder is looked up at run time, so
the .so needs no CUDA libraries on the loader path beyond the driver.  A second, small one, ``_paged.so``, is the
compiled argument marshalling of ``paged.py`` (``csrc/paged_binding.cpp``, host code against torch's headers).
"""
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libfa_sm100.so")
SOURCES = [os.path.join(HERE, "csrc", "fa_api.cu")]
HEADER = os.path.join(ROOT, "include", "fa.h")
DEPS = [os.path.join(HERE, "csrc", f) for f in os.listdir(os.path.join(HERE, "csrc")) if not f.endswith(".cpp")] + [HEADER]
BINDING = os.path.join(HERE, "_paged.so")
BINDING_SOURCE = os.path.join(HERE, "csrc", "paged_binding.cpp")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def command(verbose: bool = False):
    cmd = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
           "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "-I", os.path.join(ROOT, "include"), "-o", LIB] + SOURCES + ["-cudart", "static"]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def binding_command():
    import torch
    from torch.utils.cpp_extension import include_paths

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in include_paths()),
            f"-I{sysconfig.get_paths()['include']}", f"-I{cuda}/include", "-o", BINDING, BINDING_SOURCE, f"-L{lib}", "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch", "-ltorch_python", f"-L{HERE}", "-lfa_sm100", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]


def up_to_date(target=None, deps=None) -> bool:
    target, deps = target or LIB, deps or DEPS
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    if force or verbose or not up_to_date():
        cmd = command(verbose)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
        if verbose:
            sys.stderr.write(res.stdout + res.stderr)
    if force or not up_to_date(BINDING, [BINDING_SOURCE, HEADER]):
        cmd = binding_command()
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
