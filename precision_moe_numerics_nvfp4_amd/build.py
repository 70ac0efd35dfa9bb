"""Build libnvfp4moe.so (HIP, gfx950) in-tree, and beside it
libnvfp4moe_tensors.so (C++, what a list of torch tensors points to).

Usage: python -m precision_moe_numerics_nvfp4_amd.build [--jobs N]

Every translation unit is compiled with
  -ffp-contract=off       no fused multiply-add: every product rounds on its
                          own, as the quantization rules require;
  -fhip-fp32-correctly-rounded-divide-sqrt
                          IEEE division for the scale computations;
  -Xclang -target-feature -Xclang -packed-fp32-ops
                          keep the compiler from emitting packed-FP32 VALU
                          instructions.
"""

import argparse
import concurrent.futures as cf
import glob
import os
import shlex
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libnvfp4moe.so")
TENSORS_LIB = os.path.join(PKG, "libnvfp4moe_tensors.so")
ARCH = "gfx950"

FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"--offload-arch={ARCH}",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"),
]


def hipcc():
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found; the HIP library needs ROCm's hipcc")


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc()] + FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _build_tensors():
    """Host code against the torch that is installed (without one there are no
    tensors to look at): no GPU compiler."""
    try:
        import torch
    except ImportError:
        return
    top = os.path.dirname(torch.__file__)
    tmp = TENSORS_LIB + ".tmp"
    cmd = shlex.split(os.environ.get("CXX") or "g++") + [
        "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        "-isystem", os.path.join(top, "include"),
        "-isystem", os.path.join(top, "include", "torch", "csrc", "api", "include"),
        "-isystem", sysconfig.get_path("include"),
        os.path.join(CSRC, "tensors.cpp"), "-o", tmp,
        "-L" + os.path.join(top, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TENSORS_LIB)


def build(jobs=None, verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    jobs = jobs or min(8, len(srcs) + 1)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        tensors = ex.submit(_build_tensors)
        objs = list(ex.map(_compile, srcs))
        tensors.result()
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", f"--offload-arch={ARCH}", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}, {TENSORS_LIB}")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=None)
    a = ap.parse_args()
    build(a.jobs, verbose=True)
    sys.exit(0)
