"""Builds liblopt.so (HIP kernels + C ABI) for gfx950 in-tree, and _layers.so
(the torch calls of the norms, embedding and distillation loss).

    python -m learned_optimizer_step_amd.build
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "liblopt.so")
# (source, extra flags).  The apply kernels, and the one-launch step that
# runs them, assume finite values in their ReLUs (-fno-honor-nans gives a
# single v_max_f32 per ReLU).  The sources are compiled in parallel.
SOURCES = [("lopt_kernels.hip", []), ("lopt_apply.hip", ["-fno-honor-nans"]),
           ("lopt_single.hip", ["-fno-honor-nans"]), ("lopt_api.cpp", []), ("lopt_norm_forward.hip", []),
           ("lopt_norm_backward.hip", []), ("lopt_embedding.hip", []), ("lopt_distill.hip", []), ("lopt_ops_api.cpp", [])]
ARCH = "gfx950"

# Packed-fp32 VALU instructions are disabled for all device code.
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = ("is not a recognized feature for this target", "argument unused during compilation")
    msgs = [l for l in (res.stdout + res.stderr).splitlines() if not any(x in l for x in noise)]
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs))


def build(verbose: bool = False, out: str = LIB, defines=()) -> str:
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    cmds, objs = [], []
    for src, extra in SOURCES:
        obj = os.path.join(objdir, os.path.splitext(src)[0] + ".o")
        cmds.append([hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-c", "-Wall",
                     "-Wno-unused-function", "-I", os.path.join(ROOT, "include"), *DEVICE_FLAGS, *extra,
                     *[f"-D{d}" for d in defines],
                     os.path.join(CSRC, src), "-o", obj])
        objs.append(obj)
    with concurrent.futures.ThreadPoolExecutor(len(cmds) + 1) as ex:
        jobs = [ex.submit(_run, cmd, verbose) for cmd in cmds]
        layers = ex.submit(build_layers, verbose) if out == LIB else None
        for f in jobs:
            f.result()
        out_tmp = out + ".tmp"
        _run([hipcc(), "-shared", "-fPIC", *objs, "-o", out_tmp], verbose)
        os.replace(out_tmp, out)
    if out == LIB:
        build_microbench(verbose)
        layers.result()    # last: liblopt.so needs neither torch nor a host compiler
    return out


LAYERS = os.path.join(PKG, "_layers.so")


def _layers_object() -> str:
    return os.path.join(PKG, "_build", "layers")


def build_layers(verbose: bool = False) -> Optional[str]:
    """_layers.so from csrc/layers.cpp, for the host, against the installed torch; nothing where there is no torch."""
    import importlib.util
    if importlib.util.find_spec("torch") is None:
        print("torch is not installed: _layers.so is not built (liblopt.so does not need it)", file=sys.stderr)
        return None
    import sysconfig
    import torch
    from torch.utils import cpp_extension
    obj = _layers_object() + ".o"
    inc = [f for d in cpp_extension.include_paths() for f in ("-isystem", d)]
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    _run([cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-c", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
          "-DTORCH_EXTENSION_NAME=_layers", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc,
          "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"],
          os.path.join(CSRC, "layers.cpp"), "-o", obj], verbose)
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    # not against liblopt.so: its calls are looked up in the one that is loaded
    _run([cxx, "-shared", _layers_object() + ".o", "-L", lib, "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_hip",
          "-ldl", "-o", _layers_object() + ".so"], verbose)
    os.replace(_layers_object() + ".so", LAYERS)
    return LAYERS


MICROBENCH = os.path.join(PKG, "lopt_microbench")


def build_microbench(verbose: bool = False) -> str:
    """The machine-figure microbenchmark (read bandwidth, matrix throughput, vector-op costs)."""
    tmp = MICROBENCH + ".tmp"
    _run([hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", *DEVICE_FLAGS, "-fno-honor-nans",
          os.path.join(CSRC, "microbench.hip"), "-o", tmp], verbose)
    os.replace(tmp, MICROBENCH)
    return MICROBENCH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
