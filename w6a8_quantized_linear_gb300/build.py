"""Build libqlin.so (sm_103a) in-tree with nvcc, and the binding's short way
beside it (``_qlin_binding.so``, g++, against the headers of the torch that is
installed).

Translation units compiled in parallel (the host API with the repack
kernels, the sets of forward-kernel variants, and the kernels around the
cache and the logits), one -gencode, shared CUDA runtime (so the library and PyTorch share one runtime
and one notion of the current device).  The output goes to
``w6a8_quantized_linear_gb300/_build/libqlin.so`` (git-ignored).
"""
from __future__ import annotations

import contextlib
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libqlin.so")
BINDING = os.path.join(BUILD, "_qlin_binding.so")
STAMP = BINDING + ".torch"  # what the binding was built for; not there while a build is under way
HEADER = os.path.join(INCLUDE, "qlin.h")
UNITS = ["qlin_api.cu", "qlin_kernels_w4.cu", "qlin_kernels_w6.cu", "qlin_kernels_codebook.cu",
         "qlin_kernels_moe_w4.cu", "qlin_kernels_moe_w6.cu", "qlin_kernels_export_w4.cu", "qlin_kernels_export_w6.cu",
         "qlin_kernels_tc.cu", "qlin_kernels_tc_export.cu", "qlin_kernels_w4_one_row.cu", "qlin_kernels_w6_one_row.cu",
         "qlin_kernels_moe_one_row.cu", "qlin_kernels_codebook_one_row.cu",
         "qlin_append.cu", "qlin_attention.cu", "qlin_sample.cu", "qlin_adjust.cu",
         "qlin_evict.cu", "qlin_weigh.cu"]
SOURCES = [os.path.join(CSRC, f) for f in UNITS + ["qlin_forward.cuh", "qlin_forward_tc.cuh", "qlin_repack.cuh", "qlin_layout.h",
                                                   "qlin_ptx.cuh", "qlin_instances.h", "qlin_step.h", "qlin_tiles.cuh",
                                                   "qlin_sample_weight.h"]] + [
    HEADER]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    for cand in ("/usr/local/cuda/bin/nvcc",):
        if os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


BINDING_SOURCE = os.path.join(CSRC, "qlin_binding.cpp")


def stamp() -> str:
    """What an extension depends on beside its sources: the torch and the Python that are installed."""
    import torch
    return f"torch {torch.__version__} abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sysconfig.get_config_var('SOABI')}\n"


def binding_fits() -> bool:
    """Whether the extension was built whole, with the library that lies beside it, for this torch and Python."""
    try:
        with open(STAMP) as f:
            return f.read() == stamp()
    except OSError:
        return False


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING) or not binding_fits():
        return False

    def newer(target, sources):
        t = os.path.getmtime(target)
        return all(os.path.getmtime(s) <= t for s in sources)

    return newer(LIB, SOURCES) and newer(BINDING, [BINDING_SOURCE, HEADER])


def _torch_folder() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def _binding_command(obj: str) -> list:
    import torch
    inc = os.path.join(_torch_folder(), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", inc, "-isystem",
            os.path.join(inc, "torch", "csrc", "api", "include"), "-c", BINDING_SOURCE, "-o", obj]


def _link_binding(obj: str, tag: str) -> str:
    lib = os.path.join(_torch_folder(), "lib")
    tmp = BINDING + tag
    r = subprocess.run(["g++", "-shared", obj, "-o", tmp, "-L", BUILD, "-l:libqlin.so", "-L", lib, "-ltorch_python", "-ltorch_cpu",
                        "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("linking the binding failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, BINDING)
    return r.stdout + r.stderr


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = nvcc_path()
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
    tag = f".tmp{os.getpid()}"
    # kernels are instantiated in one unit and launched from another, so their
    # host stubs need external linkage
    common = [nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo", "-O3", "-std=c++17",
              "-static-global-template-stub=false", "-Xcompiler", "-fPIC", "-I", INCLUDE]
    if verbose:
        common.insert(1, "-Xptxas=-v")
    objs, procs = [], []
    try:
        return _compile_and_link(nvcc, cuda_lib, common, tag, verbose)
    finally:
        for f in os.listdir(BUILD):  # objects of this build, also after a failure
            if f.endswith(tag + ".o"):
                os.remove(os.path.join(BUILD, f))


def _compile_and_link(nvcc, cuda_lib, common, tag, verbose):
    objs, procs = [], []
    for u in UNITS:
        obj = os.path.join(BUILD, u.replace(".cu", tag + ".o"))
        cmd = common + ["-c", os.path.join(CSRC, u), "-o", obj]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        objs.append(obj)
    binding = os.path.join(BUILD, "qlin_binding" + tag + ".o")
    cmd = _binding_command(binding)
    procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    logs = []
    for cmd, pr in procs:
        out, _ = pr.communicate()
        logs.append(out)
        if pr.returncode != 0:
            raise RuntimeError("compiling failed:\n" + " ".join(cmd) + "\n" + out)
    tmp = LIB + tag
    cmd = [nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-cudart", "shared", "-Xlinker",
           f"-rpath,{cuda_lib}"] + objs + ["-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    with contextlib.suppress(FileNotFoundError):  # (also where another process's build has just removed it)
        os.remove(STAMP)
    os.replace(tmp, LIB)
    logs.append(_link_binding(binding, tag))
    with open(STAMP + tag, "w") as f:
        f.write(stamp())
    os.replace(STAMP + tag, STAMP)
    if verbose:
        print("".join(logs) + r.stdout + r.stderr)
    return LIB


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
