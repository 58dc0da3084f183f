"""Build ``libnvfp4.so`` (the CUDA library behind include/nvfp4.h) in-tree with nvcc.

Only sm_103a is targeted. Translation units compile in parallel, then link into one shared
library with the CUDA runtime linked statically (the driver is reached through the runtime).
"""
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libnvfp4.so")
SOURCES = ["quantize_row.cu", "quantize_col.cu", "quantize_rowcol.cu", "quantize_rowcol_rht.cu",
           "quantize_rowcol_rht_fast.cu",
           "quantize_2d.cu", "amax_dequant.cu", "nvfp4_api.cu", "quantize_noalloc.cu",
           "host_pipeline.cu", "amax_pass.cu", "mx_kernel.cu", "producer.cu",
           "moe_route.cu", "checkpoint.cu", "moe_checkpoint_api.cu",
           "router.cu", "gemm.cu", "gemm_epilogue.cu", "gemm_api.cu", "adamw.cu"]
HEADERS = ["nvfp4_device.cuh", "nvfp4_internal.h", "aux_internal.h", "quantize_kernel.cuh",
           "fused_amax.cuh", "tile_ring.h", "gemm_internal.h", "gemm_device.cuh",
           "tcgen05.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-fmad=false",                     # no multiply-add contraction outside explicit fma
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libnvfp4")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "nvfp4.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile if sources changed (or force); return the library path."""
    if not force and not _stale():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    pid = os.getpid()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".%d.o" % pid))
        cmd = [nvcc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp.%d" % pid
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    for o in objs:
        os.remove(o)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
