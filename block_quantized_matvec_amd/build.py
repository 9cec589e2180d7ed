"""Build libft.so (the gfx950 HIP kernels + C ABI) in-tree with hipcc, and _ft_bind.so (marshalling of the smallest
calls, against torch's headers) with g++.

    python -m block_quantized_matvec_amd.build

Always recompiles.  Translation units compile in parallel; the shared objects are
written next to this file so that they travel with the source tree.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libft.so")
BIND = os.path.join(PKG, "_ft_bind.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["ft_mmvq_kq.hip", "ft_mmvq_kq_b.hip", "ft_mmvq_kq_c.hip", "ft_mmvq_kq_d.hip", "ft_mmvq_q8k.hip", "ft_mmvq.hip",
           "ft_api.cpp", "ft_quant.hip", "ft_mmvq_mfma.hip", "ft_moe.hip", "ft_moe_fused.hip", "ft_moe_fp4.hip", "ft_grouped.hip",
           "ft_probe.hip", "ft_kv.hip", "ft_attn.hip", "ft_attn_d64.hip", "ft_attn_d96.hip", "ft_attn_d128.hip",
           "ft_attn_d256.hip", "ft_route.hip", "ft_rope.hip", "ft_norm.hip", "ft_lora.hip"]

CFLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # no packed-fp32 VALU ops: the compiler must not form v_pk_{add,mul,fma}_f32
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # IEEE fp32 divide (the quantizers decide integers from x/d)
    "-fhip-fp32-correctly-rounded-divide-sqrt", "-fno-fast-math", "-ffp-contract=fast",
    # MFMA results in VGPRs (no AGPR copies back for the integer scale combine)
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wall", "-Wno-unused-function", "-Wno-unused-variable",
    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
]

# every fp32 operation rounded by itself (the quantized code of a normed or turned element hangs on no pairing)
EXTRA = {"ft_rope.hip": ["-ffp-contract=off"], "ft_norm.hip": ["-ffp-contract=off"]}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    cmd = [HIPCC] + CFLAGS + EXTRA.get(src, []) + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    warn = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l and l.strip())
    if warn and "warning" in warn:
        sys.stderr.write(warn + "\n")
    return obj


def _bind() -> None:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    tmp = BIND + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           "-I" + os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-isystem", "/opt/rocm/include",
           os.path.join(CSRC, "ft_bind.cpp"), "-o", tmp, "-L" + os.path.join(torch, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for ft_bind.cpp:\n{r.stdout}\n{r.stderr}")
    if "warning" in r.stderr:
        sys.stderr.write(r.stderr + "\n")
    os.replace(tmp, BIND)


def build(jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES), max(1, min(os.cpu_count() or 2, 16)))
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _bind()
    return LIB


if __name__ == "__main__":
    print(build())
