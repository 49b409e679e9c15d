"""Build libnf4.so in-tree with hipcc for gfx950, and the compiled part of its
Python binding (_nf4_torch, host code against torch's headers).

Run as `python -m nf4_bit_weight_amd.build` or through __graft_entry__.build().
Each .hip file compiles to an object in parallel; the objects link into
nf4_bit_weight_amd/libnf4.so, which the ctypes binding loads.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libnf4.so")
ARCH = "gfx950"

SOURCES = ("nf4_abi.hip", "nf4_codec.hip", "nf4_gemm.hip", "nf4_gemv.hip", "nf4_attn_abi.hip",
           "nf4_kv.hip", "nf4_prompt.hip", "nf4_experts_abi.hip", "nf4_experts.hip", "nf4_int8.hip")

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # single rounding for every fp32 op of the codec (no multiply-add contraction)
    "-ffp-contract=off",
    # packed fp32 VALU ops are kept out of the generated code on this target
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
    "-Wno-unused-result",
]


TORCH_SOURCES = ("nf4_torch.cpp", "nf4_torch_experts.cpp")
TORCH_LIB = os.path.join(PKG, "_nf4_torch.so")


def torch_module_cmds(objs):
    """(one compile of each source, link) of the binding module: plain host C++."""
    import sysconfig

    import torch

    base = os.path.dirname(os.path.abspath(torch.__file__))
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    inc = [os.path.join(base, "include"), sysconfig.get_paths()["include"], os.path.join(rocm, "include")]
    compile_ = [["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                *[f for d in inc for f in ("-isystem", d)], "-c", os.path.join(CSRC, src), "-o", obj]
                for src, obj in zip(TORCH_SOURCES, objs)]
    lib = os.path.join(base, "lib")
    link = ["g++", "-shared", "-fPIC", *objs, "-L", PKG, "-l:libnf4.so", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
            "-lc10_hip", "-Wl,-rpath,$ORIGIN", "-o", TORCH_LIB + ".tmp"]
    return compile_, link


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libnf4.so)")


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = hipcc()
    procs = []
    objs = []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        if not os.path.exists(path):
            continue
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        objs.append(obj)
        cmd = [cc, *HIPCC_FLAGS, "-c", path, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    torch_compile, torch_link = torch_module_cmds([os.path.join(BUILD_DIR, s.replace(".cpp", ".o")) for s in TORCH_SOURCES])
    for src, cmd in zip(TORCH_SOURCES, torch_compile):
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        # the host pass does not know the packed-fp32 feature name; that note is harmless
        lines = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln]
        if p.returncode != 0:
            failed.append(src)
            print("\n".join(lines), file=sys.stderr)
        elif verbose and lines:
            print("\n".join(lines))
    if failed:
        raise RuntimeError(f"compilation failed for {failed}")
    tmp = LIB + ".tmp"
    link = [cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        print(r.stdout.decode(errors="replace"), file=sys.stderr)
        raise RuntimeError("link of libnf4.so failed")
    os.replace(tmp, LIB)
    r = subprocess.run(torch_link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        print(r.stdout.decode(errors="replace"), file=sys.stderr)
        raise RuntimeError("link of _nf4_torch.so failed")
    os.replace(TORCH_LIB + ".tmp", TORCH_LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
