"""Builds libpnq.so in-tree (one nvcc process per translation unit, in parallel, for sm_103a) and, where torch and g++ are
there, _native.so beside it, the torch wrappers of the 4-bit operands and the expert layer. The C library needs nvcc alone."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libpnq.so")
NATIVE = os.path.join(PKG, "_native.so")
BUILD_DIR = os.path.join(ROOT, "_build")
SOURCES = ["pnq_api.cu", "pnq_codec_kernels.cu", "pnq_gemv_simt.cu", "pnq_gemv_pn.cu", "pnq_gemv_nvfp4.cu",
           "pnq_grouped.cu", "pnq_quantize.cu", "pnq_prefill.cu", "pnq_fp4_api.cu", "pnq_fp4_quantize.cu",
           "pnq_fp4_gemm.cu", "pnq_experts.cu", "pnq_norm.cu", "pnq_route.cu", "pnq_int8_gemm.cu", "pnq_int8_mma.cu", "pnq_int8_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libpnq.so")
    return path


def _cuda_lib_dir(nv: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nv))), "lib64")


def _deps(src: str) -> list[str]:
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + \
        [os.path.join(INCLUDE, "pnq.h"), src]


def _torch_dir() -> str | None:
    """Where the installed torch is, None where there is none."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    return list(spec.submodule_search_locations)[0]


def _native_compile(nv: str, torch_dir: str):
    """The compile command of pnq_torch.cpp, or None where its object is up to date for this torch and Python."""
    src, obj, stamp = (os.path.join(CSRC, "pnq_torch.cpp"), os.path.join(BUILD_DIR, "pnq_torch.o"),
                       os.path.join(BUILD_DIR, "pnq_torch.stamp"))
    with open(os.path.join(torch_dir, "version.py")) as f:
        key = torch_dir + "\n" + f.read() + sysconfig.get_config_var("EXT_SUFFIX")
    have = open(stamp).read() if os.path.exists(stamp) else None
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "pnq.h")))
    if have == key and os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return None
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nv))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE, "-isystem", os.path.join(torch_dir, "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda_include, "-c", src, "-o", obj]
    return cmd, stamp, key


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    nv = nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = ["-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC", "-I", CSRC, "-I", INCLUDE,
             "--expt-relaxed-constexpr"] + (extra_flags or [])
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(d) for d in _deps(s)):
            jobs.append([nv, *flags, "-c", s, "-o", o])
    torch_dir = _torch_dir()
    wrappers = torch_dir is not None and shutil.which("g++") is not None
    if not wrappers:
        print(f"{'torch' if torch_dir is None else 'g++'} not found: building {os.path.basename(LIB)} without the torch wrappers of "
              "the 4-bit operands, the expert layer, the norms and the 8-bit rows and product")
    native = _native_compile(nv, torch_dir) if wrappers else None
    if native is not None:
        jobs.append(native[0])
    if verbose:
        for j in jobs:
            print(" ".join(j))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        results = list(ex.map(lambda cmd: subprocess.run(cmd, capture_output=True, text=True), jobs))
    failed = None  # of the wrappers' compile: raised once the C library is there
    for cmd, r in zip(jobs, results):
        if r.returncode != 0:
            failed = RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
            if native is None or cmd is not native[0]:
                raise failed
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
    objs = [os.path.join(BUILD_DIR, s.replace(".cu", ".o")) for s in SOURCES]
    if force or jobs or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        libdir = _cuda_lib_dir(nv)
        cmd = [nv, "-shared", *ARCH, "-cudart", "shared", "-o", tmp, *objs,
               "-Xlinker", f"-rpath,{libdir}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if failed is not None:
        raise failed
    if wrappers and (jobs or force or not os.path.exists(NATIVE)):
        torch_lib = os.path.join(torch_dir, "lib")
        tmp = NATIVE + f".tmp{os.getpid()}"
        cmd = ["g++", "-shared", "-o", tmp, os.path.join(BUILD_DIR, "pnq_torch.o"), "-L", PKG, "-l:libpnq.so", "-L", torch_lib, "-lc10",
               "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, NATIVE)
        if native is not None:
            with open(native[1], "w") as f:
                f.write(native[2])
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
