"""Build ``libsdv.so`` (the CUDA path, sm_103a) in-tree with nvcc.

Each translation unit compiles in parallel to an object under
``draft_verification_sdv_gb300/_build/``; the objects link into
``draft_verification_sdv_gb300/libsdv.so``.  Plain IEEE arithmetic (no
fast-math); ``-lineinfo`` for profiling.
"""
import concurrent.futures
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libsdv.so")
SOURCES = ["k1_rowpass.cu", "k2_select.cu", "k3_sample.cu", "k4_cps.cu", "k5_adl.cu", "k6_rope.cu", "k7_kvcache.cu",
           "k8_attn.cu", "k8_attn_tc.cu", "k8_attn_dec.cu", "k8_attn_mma64.cu", "k8_attn_mma128.cu", "k8_attn_mma256.cu", "k9_logits.cu", "k10_tree.cu",
           "sdv_api.cu", "sdv_layer.cu", "sdv_static.cu"]
HEADERS = ["sdv_device.cuh", "sdv_plan.h", "sdv_layer.h", "k8_attn.cuh", "k8_attn_mma.cuh", "k8_attn_tma.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# Kernels that exchange registers between their warps need a launch with just this
# many per thread (kRegs of the source): with another count every call is refused.
REGISTERS = {"k8_attn_tc.cu": ("attn_tc_kernel", 168)}


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    return ([os.path.join(CSRC, f) for f in SOURCES + HEADERS]
            + [os.path.join(ROOT, "include", "sdv.h"), os.path.abspath(__file__)])


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("command failed: %s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
    return r.stdout + r.stderr


def check_registers(src: str, report: str) -> None:
    """Raise unless the compiler's report (-Xptxas -v) of `src` gives each kernel
    of REGISTERS its count."""
    kernel, want = REGISTERS[src]
    found = re.findall(r"Compiling entry function '(\S*)'.*?Used (\d+) registers", report, re.S)
    counts = [int(n) for name, n in found if kernel in name]
    if not counts or set(counts) != {want}:
        raise RuntimeError("%s: %s must have %d registers per thread, the compiler gave %s"
                           % (src, kernel, want, counts))


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile libsdv.so if any source is newer than it; return its path."""
    if not force and os.path.exists(LIB) and all(
            os.path.getmtime(LIB) >= os.path.getmtime(d) for d in _deps()):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nv = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", os.path.join(ROOT, "include")]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        report = ["-Xptxas", "-v"] if src in REGISTERS and not verbose_ptxas else []
        out = _run([nv] + flags + report + ["-c", os.path.join(CSRC, src), "-o", obj])
        if src in REGISTERS:
            check_registers(src, out)
        return obj, out

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose_ptxas:
        for _, out in results:
            sys.stdout.write(out)
    tmp = LIB + ".tmp"
    _run([nv] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + ["-lcudart"])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
