"""Builds the CUDA library in-tree: moe_expert_layer_gb300/_build/libmoe_layer.so.

Each translation unit under csrc/ is compiled for sm_103a in parallel, then the
objects are linked into one shared library (CUDA runtime linked statically).
"""
import concurrent.futures as cf
import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libmoe_layer.so")
SOURCES = ["route_sort.cu", "elementwise.cu", "gemm_hmma.cu", "gemm_tc.cu", "gemm_dispatch.cu", "moe_layer.cu",
           "route_sort_noalloc.cu", "selftest.cu", "weight_tiles.cu",
           "route_topk.cu", "mxfp4_quant.cu", "mxfp4_gmm.cu", "mxfp4_few.cu",
           "mxfp4_abi.cu",
           "rows16.cu", "gmm16.cu", "lora16.cu", "experts16_abi.cu"]
HEADERS = ["abi_checks.h", "common.cuh", "experts16.h", "kernels.h", "mx_tc.cuh", "mxfp4.cuh", "mxfp4.h", "swiglu.cuh", "tc_common.cuh",
           "tensor_map.h"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else "nvcc")
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]
# Kernels whose warps hand registers over to one another (setmaxnreg), by source and mangled name, and the registers
# a thread has to be launched with: with fewer they would wait for ones that are not there, so such a build is refused
# here.  The weight gradients of gmm16.cu whose sums are in parts (Sums::kFewParts, kParts).
LAUNCH_REGISTERS = {"gmm16.cu": (r"gmm16_kernel\w*SumsE[23]E", 2, 168)}


def _inputs():
    root = os.path.dirname(HERE)
    return ([os.path.join(CSRC, s) for s in SOURCES + HEADERS]
            + [os.path.join(root, "include", h) for h in ("moe_layer.h", "moe_mxfp4.h", "moe_experts16.h")] + [os.path.abspath(__file__)])


def check_registers(src, log):
    """Raises unless the kernels of LAUNCH_REGISTERS in this source are there and have their registers, by what
    ptxas -v says of them."""
    pattern, kernels, wanted = LAUNCH_REGISTERS[src]
    found = re.findall(r"Compiling entry function '(\w+)'(?:(?!Compiling entry).)*?Used (\d+) registers", log, re.S)
    got = [int(n) for name, n in found if re.search(pattern, name)]
    if got != [wanted] * kernels:
        raise RuntimeError("%s: %d kernels /%s/ of %d registers wanted, built with %s"
                           % (src, kernels, pattern, wanted, got))


def up_to_date():
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build(force=False, verbose=False):
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        flags = ["-Xptxas", "-v"] if src in LAUNCH_REGISTERS else []
        cmd = [NVCC] + NVCC_FLAGS + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if flags:
            check_registers(src, r.stdout + r.stderr)
        elif verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [NVCC, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
