"""Build libexq.so in-tree: host code with g++ (OpenMP), kernels with hipcc for gfx950; and _exq_torch.so, the calls on
PyTorch tensors, with g++ against PyTorch's headers (where PyTorch is installed)."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libexq.so")
BUILD_DIR = os.path.join(ROOT, "_build")

HIP_SOURCES = ("exq_device.hip", "exq_prefill.hip", "exq_cache.hip", "exq_pages.hip", "exq_rotate.hip", "exq_lora.hip",
               "exq_sample.hip")
HOST_SOURCES = ("exq_host.cpp",)
TORCH_SOURCE = "exq_torch.cpp"
TORCH_LIB = os.path.join(PKG, "_exq_torch.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17",
    # no packed fp32 instructions anywhere in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines() if "not a recognized feature" not in l)
    if r.returncode != 0:
        sys.stderr.write(out + "\n")
        raise RuntimeError("build step failed: " + " ".join(cmd))
    return out


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def _torch_flags():
    """(compile flags, link flags) of an extension module on PyTorch tensors; None without PyTorch."""
    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError:
        return None
    includes = cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]
    compile_flags = ["-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
    for path in includes:
        compile_flags += ["-isystem", path]
    return compile_flags, ["-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"]


def build(verbose: bool = False) -> str:
    """Compile every source (always, all at once) and link libexq.so and _exq_torch.so next to this file.

    The library needs neither PyTorch nor Python's headers: if the extension fails, it is linked before the error is raised."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = []
    for src in HOST_SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        jobs.append((obj, ["g++", "-O2", "-fPIC", "-fopenmp", "-std=c++17", "-ffp-contract=off", "-Wall",
                           "-c", os.path.join(CSRC, src), "-o", obj]))
    for src in HIP_SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        jobs.append((obj, [hipcc()] + HIPCC_FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]))
    torch_flags = _torch_flags()
    torch_obj = os.path.join(BUILD_DIR, TORCH_SOURCE + ".o")
    lib_objs = [o for o, _ in jobs]
    if torch_flags:
        jobs.append((torch_obj, ["g++", "-O2", "-fPIC", "-std=c++17", "-Wall"] + torch_flags[0] +
                     ["-c", os.path.join(CSRC, TORCH_SOURCE), "-o", torch_obj]))
    procs = [(cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
             for _, cmd in jobs]
    failed = {}   # by object: the command
    for (obj, cmd), (_, p) in zip(jobs, procs):
        out = "\n".join(l for l in p.communicate()[0].splitlines() if "not a recognized feature" not in l)
        if p.returncode != 0:
            sys.stderr.write(out + "\n")
            failed[obj] = cmd
        elif verbose and out.strip():
            print(out)

    def check(objs):
        for obj in objs:
            if obj in failed:
                raise RuntimeError("build step failed: " + " ".join(failed[obj]))

    check(lib_objs)
    tmp = LIB + ".tmp%d" % os.getpid()
    _run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + lib_objs + ["-lgomp"])
    os.replace(tmp, LIB)
    if torch_flags:
        check([torch_obj])
        tmp = TORCH_LIB + ".tmp%d" % os.getpid()
        _run(["g++", "-shared", "-fPIC", "-o", tmp, torch_obj, "-L" + PKG, "-l:" + os.path.basename(LIB),
              "-Wl,-rpath,$ORIGIN"] + torch_flags[1])
        os.replace(tmp, TORCH_LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
