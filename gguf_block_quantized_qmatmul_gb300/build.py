"""Build the CUDA library (libqmm.so) in-tree with nvcc for sm_103a.

Translation units are compiled in parallel and linked into
``gguf_block_quantized_qmatmul_gb300/_build/libqmm.so``.  No fast-math flags:
the quantizers rely on IEEE round-to-nearest intrinsics.  Beside it the host
compiler builds ``_qmm_torch.so``, the CPython extension that q4g.py calls.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libqmm.so")
BINDING = os.path.join(BUILD, "_qmm_torch.so")  # CPython extension of q4g.py's calls
ROOT = os.path.dirname(HERE)
UNITS = ["qmm_api", "qmm_quant", "qmm_stream_q8_0", "qmm_stream_q4_k", "qmm_stream_x_0", "qmm_stream_q6_k", "qmm_gemv_q8_0", "qmm_gemv_q4_k", "qmm_dmma", "qmm_dmma_x_0", "qmm_dmma_q6_k", "qmm_tc", "qmm_tcx", "qmm_tcx_f32", "qmm_static_ws", "qmm_batch", "qmm_batch_mix", "qmm_q4g_api", "qmm_q4g_layout", "qmm_q4g_rows", "qmm_q4g_rows_1", "qmm_q4g_rows_2", "qmm_q4g_rows_4",
         "qmm_q4g_gemm", "qmm_moe_route"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqmm.so")


def _deps():
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    out.append(os.path.join(ROOT, "include", "qmm.h"))
    out.append(os.path.abspath(__file__))
    return out


def _binding_command(out: str, lib_dir: str) -> list[str]:
    """Host compiler command for the CPython extension, linked against this torch and the libqmm.so of lib_dir."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *(f"-I{i}" for i in inc),
            os.path.join(CSRC, "qmm_torch.cpp"), "-o", out, f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch",
            "-ltorch_python", f"-Wl,-rpath,{lib}", f"-L{lib_dir}", "-Wl,--no-as-needed", "-l:libqmm.so", "-Wl,-rpath,$ORIGIN"]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    procs = []
    # Libraries are made in a folder of their own and moved to their places when all are whole: what other processes
    # load, and what up_to_date() sees, is the last build's or this one's.
    with tempfile.TemporaryDirectory(prefix="link.", dir=BUILD) as tmp:
        try:
            for u in UNITS:
                obj = os.path.join(tmp, u + ".o")
                log = open(os.path.join(BUILD, u + ".ptxas.txt"), "w")
                cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, u + ".cu"), "-o", obj]
                procs.append((u, subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT), log))
            # the extension needs libqmm.so's name only: it is linked against an empty one while that compiles
            stub, binding, lib = os.path.join(tmp, "stub"), os.path.join(tmp, "binding.so"), os.path.join(tmp, "lib.so")
            os.mkdir(stub)
            subprocess.run([os.environ.get("CXX", "g++"), "-shared", "-fPIC", "-x", "c++", "/dev/null", "-o", os.path.join(stub, "libqmm.so")], check=True)
            log = open(os.path.join(BUILD, "qmm_torch.ptxas.txt"), "w")
            procs.append(("qmm_torch", subprocess.Popen(_binding_command(binding, stub), stdout=log, stderr=subprocess.STDOUT), log))
            failed = [u for u, p, _ in procs if p.wait() != 0]
        finally:
            for _, p, log in procs:
                if p.poll() is None:
                    p.kill()
                    p.wait()
                log.close()
        if failed:
            msgs = "".join(open(os.path.join(BUILD, u + ".ptxas.txt")).read()[-4000:] for u in failed)
            raise RuntimeError(f"nvcc failed for {failed}:\n{msgs}")
        subprocess.run([nvcc, *ARCH, "-shared", "-o", lib] + [os.path.join(tmp, u + ".o") for u in UNITS], check=True)
        os.replace(lib, LIB)
        os.replace(binding, BINDING)
    for f in (LIB, BINDING):
        os.utime(f)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
