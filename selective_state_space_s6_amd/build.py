"""Build libssmscan.so (gfx950) from the HIP sources in csrc/, and _attn_bind.so, the
compiled part of the Python binding (host code only, against torch's headers).

Usage: python selective_state_space_s6_amd/build.py   (or __graft_entry__.build())
Each source is compiled to an object in parallel, then linked into a shared
library next to this file.  Always recompiles (no staleness heuristics).
libssmscan.so needs hipcc alone and is linked first; where torch is not installed it is all
that is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libssmscan.so")
BIND = os.path.join(HERE, "_attn_bind.so")
SOURCES = ["abi.hip", "s6_scan.hip", "s6_seg.hip", "s6_fused.hip", "s6_decode.hip", "s6_bwd.hip", "ssd_scan.hip", "ssd_decode.hip", "ssd_bwd.hip", "cssd_scan.hip",
           "trap_rotate.hip", "conv1d.hip", "s6_grouped.hip", "scratch.hip",
           "abi_attn.hip", "kv_pages.hip", "qk_rope.hip", "paged_attn.hip"]
ARCH = os.environ.get("SSM_OFFLOAD_ARCH", "gfx950")
# Packed fp32 ops are switched off: the compiler must not emit v_pk_{add,mul,fma}_f32.
# MFMA accumulators are kept in ordinary VGPRs, so the fp32 state that the SSD
# kernels scale and split between contractions needs no AGPR round trips.
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-I", INCLUDE,
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-mllvm", "-amdgpu-mfma-vgpr-form=1",
          "-Wno-unused-command-line-argument"]


def _hipcc() -> str:
    for c in ("/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def _compile(src: str, obj: str) -> None:
    cmd = [_hipcc(), *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")


def _compile_bind(obj: str) -> None:
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", "/opt/rocm/include",
           "-I", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "bind_attn.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for bind_attn.cpp:\n{r.stdout}\n{r.stderr}")


def _link_bind(obj: str) -> None:
    import torch
    cmd = ["g++", "-shared", "-o", BIND + ".tmp", obj, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
           "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python", "-L", HERE, "-l:libssmscan.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _attn_bind.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(BIND + ".tmp", BIND)


def build(verbose: bool = True) -> str:
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = [os.path.join(objdir, s.replace(".hip", ".o")) for s in SOURCES]
    bind_obj = os.path.join(objdir, "bind_attn.o")
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        bind = ex.submit(_compile_bind, bind_obj) if importlib.util.find_spec("torch") else None
        list(ex.map(lambda so: _compile(*so), zip(SOURCES, objs)))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if bind:
        bind.result()
        _link_bind(bind_obj)
    if verbose:
        print(f"built {LIB}, " + (BIND if bind else "and no _attn_bind.so: torch is not installed"))
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
