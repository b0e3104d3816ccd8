"""Build libkda.so in-tree for gfx950 with hipcc.

    python -m gated_delta_rule_51_amd.build

Every .hip file under csrc/ is compiled to an object under _build/ (in
parallel), then linked into gated_delta_rule_51_amd/libkda.so; csrc/binding.cpp
(host code over torch's headers) becomes gated_delta_rule_51_amd/_binding.so.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libkda.so")
BINDING = os.path.join(PKG, "_binding.so")
BUILD = os.path.join(ROOT, "_build")

ARCH = "gfx950"
FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "--offload-arch=" + ARCH,
    # never emit packed fp32 instructions (v_pk_{add,mul,fma}_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc()] + FLAGS + ["-I", CSRC, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, r.stderr))
    return obj


def _compile_binding() -> str:
    import torch
    from torch.utils.cpp_extension import include_paths
    cxx = shutil.which("g++") or shutil.which("c++") or hipcc()
    obj = os.path.join(BUILD, "binding.cpp.o")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"]]
    for path in include_paths():
        cmd += ["-isystem", path]
    r = subprocess.run(cmd + ["-c", os.path.join(CSRC, "binding.cpp"), "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the binding failed to compile:\n%s" % r.stderr)
    return obj


def _link_binding(obj: str) -> None:
    import torch
    cxx = shutil.which("g++") or shutil.which("c++") or hipcc()
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [cxx, "-shared", "-fPIC", "-o", tmp, obj, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python",
           "-ltorch_cpu", "-ltorch", "-lc10", "-L", PKG, "-lkda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("the binding failed to link:\n%s" % r.stderr)
    os.replace(tmp, BINDING)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, srcs))
    tmp = OUT + ".tmp%d" % os.getpid()
    cmd = [hipcc(), "-shared", "-fPIC", "--offload-arch=" + ARCH, "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s" % r.stderr)
    os.replace(tmp, OUT)
    _link_binding(binding.result())   # the C library is there, whatever the binding lacks
    if verbose:
        print("built", OUT, "and", BINDING)
    return OUT


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
