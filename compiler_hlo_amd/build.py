"""Build the hero-fusion library (libhlofusion.so) in-tree.

The host library (planner, code generator, hiprtc driver, C ABI) is plain C++
compiled with g++ against the HIP runtime and hiprtc; the one device array the
library holds itself (the no-allocation launch's scratch memory) and the
operators' kernels are compiled with hipcc for gfx950 and linked in.  The hand-written
device templates under csrc/kernels are embedded into it as text; every
fusion's kernel is generated from them and compiled for gfx950 by hiprtc at
hf_fusion_create time.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
KERNELS = os.path.join(CSRC, "kernels")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libhlofusion.so")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
TEMPLATES = ["common", "loop", "transpose", "reduce_row", "reduce_col"]
SOURCES = ["intake.cpp", "plan.cpp", "codegen.cpp", "hlofusion.cpp", "operators/operators.cpp"]


def embed() -> str:
    os.makedirs(BUILD, exist_ok=True)
    out = os.path.join(BUILD, "kernels_embed.inc")
    parts = ["// generated by compiler_hlo_amd/build.py from csrc/kernels/*.hip\n"]
    for name in TEMPLATES:
        text = open(os.path.join(KERNELS, name + ".hip")).read()
        assert ")HFK\"" not in text
        parts.append('static const char k_src_%s[] = R"HFK(%s)HFK";\n' % (name, text))
    data = "".join(parts)
    if not os.path.exists(out) or open(out).read() != data:
        with open(out, "w") as f:
            f.write(data)
    return out


# Device code compiled into the library itself (the no-allocation launch's
# scratch array, the operators' kernels); compiled with hipcc for gfx950,
# without packed FP32, one process a file.
HIP_SOURCES = ["scratch.hip", "operators/rows.hip", "operators/experts.hip", "operators/product.hip",
               "operators/product_experts.hip", "operators/product_experts_grad.hip", "operators/skinny.hip"]
HIPCC_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def build(verbose: bool = False) -> str:
    embed()
    tmp = LIB + ".tmp%d" % os.getpid()
    objs, running = [], []
    for src in HIP_SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        hcmd = [os.path.join(ROCM, "bin", "hipcc")] + HIPCC_FLAGS + [
            "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(hcmd), flush=True)
        running.append((hcmd, subprocess.Popen(hcmd)))
        objs.append(obj)
    failed = [subprocess.CalledProcessError(p.returncode, c) for c, p in running if p.wait() != 0]
    if failed:
        raise failed[0]
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-Wextra",
           "-Wno-unused-parameter", "-D__HIP_PLATFORM_AMD__",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", BUILD,
           "-I", os.path.join(ROCM, "include")]
    cmd += [os.path.join(CSRC, s) for s in SOURCES] + objs
    cmd += ["-o", tmp, "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-lhiprtc",
            "-Wl,-rpath," + os.path.join(ROCM, "lib")]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
