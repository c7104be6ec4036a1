"""Builds ``libssmscan.so`` in-tree: hipcc for the gfx950 kernels, g++ for the
C-ABI layer, linked against the HIP runtime; and ``_ssmtensors.so``, the module
with which the binding reads lists of tensors (g++, against Python and torch).

Every compile recompiles (no staleness heuristics): ``build()`` is the "does
it build" step.  ``ensure_built()`` builds only when one of the two is missing.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libssmscan.so")
TENSORS = os.path.join(PKG, "_ssmtensors.so")
BUILD_DIR = os.path.join(PKG, "_build")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
ARCH = "gfx950"

# Packed-FP32 VALU forms are disabled for all device code.
HIP_FLAGS = ["-O3", "-std=c++17", "-fPIC", "--offload-arch=" + ARCH,
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-ffp-contract=fast", "-munsafe-fp-atomics", "-Wall"]


def _finish(cmd, proc):
    out, _ = proc.communicate()
    out = "\n".join(l for l in out.splitlines()
                    if "packed-fp32-ops" not in l and "--hip-link" not in l)
    if proc.returncode != 0:
        sys.stderr.write(out + "\n")
        raise RuntimeError("build step failed: " + " ".join(cmd))
    return out


def _start(cmd):
    return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                 stderr=subprocess.STDOUT, text=True)


def _run(cmd):
    return _finish(*_start(cmd))


HIP_SOURCES = ["ssm_kernels.hip", "ssm_step.hip", "ssm_bwd.hip", "ssm_ssd.hip",
               "ssm_roofline.hip", "ssm_conv_bwd.hip", "ssm_linattn.hip",
               "ssm_linattn_out_bf16.hip", "ssm_linattn_out_f32.hip",
               "ssm_linattn_grads_bf16.hip", "ssm_linattn_grads_f32.hip",
               "ssm_block_norm.hip", "ssm_embed.hip", "ssm_layer_norm.hip",
               "ssm_grad.hip"]
CPP_SOURCES = ["ssm_api.cpp", "ssm_linattn_api.cpp", "ssm_model_api.cpp"]


def _tensors_command(out):
    """The module of lists of tensors, which only the binding loads: torch's
    libraries are in the process by then."""
    import torch
    base = os.path.dirname(torch.__file__)
    include = os.path.join(base, "include")
    system = [include, os.path.join(include, "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"]]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wextra",
             "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi(), "-I", INCLUDE]
            + [a for d in system for a in ("-isystem", d)]
            + [os.path.join(CSRC, "ssm_tensors.cpp"), "-o", out,
               "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"])


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    hipcc = os.path.join(ROCM, "bin", "hipcc")
    objs = []
    jobs = []
    for src in HIP_SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        objs.append(obj)
        jobs.append(_start([hipcc] + HIP_FLAGS + ["-I", INCLUDE, "-I", CSRC, "-c",
                                                  os.path.join(CSRC, src), "-o", obj]))
    for src in CPP_SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cpp", ".o"))
        objs.append(obj)
        jobs.append(_start(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wextra",
                            "-I", INCLUDE, "-I", CSRC, "-c",
                            os.path.join(CSRC, src), "-o", obj]))
    tensors = TENSORS + ".tmp%d" % os.getpid()
    jobs.append(_start(_tensors_command(tensors)))
    out = "".join(_finish(*j) for j in jobs)
    tmp = LIB + ".tmp%d" % os.getpid()
    out += _run([hipcc, "-shared", "-fPIC", "--offload-arch=" + ARCH, "-o", tmp]
                + objs + ["-L", os.path.join(ROCM, "lib"), "-lamdhip64",
                          "-Wl,-rpath," + os.path.join(ROCM, "lib")])
    os.replace(tensors, TENSORS)
    os.replace(tmp, LIB)
    if verbose and out.strip():
        print(out)
    return LIB


def ensure_built() -> str:
    if not (os.path.exists(LIB) and os.path.exists(TENSORS)):
        build()
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
