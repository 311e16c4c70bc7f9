"""A C program whose host memory has run out: every allocation of the process throws std::bad_alloc when the library's calls come.
They answer PNQ_ERR_CUDA (no exception leaves a C entry, which would end the process), and work once there is memory again."""
import os
import shutil
import subprocess

import pytest

import block_quantized_weight_pn3t_gb300 as pnq

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLIENT = r"""
#include <cuda_runtime.h>
#include <cstdio>
#include <cstdlib>
#include <new>
#include "pnq.h"

static bool none_left = false;
void* operator new(std::size_t n) {
    void* p = none_left ? nullptr : std::malloc(n ? n : 1);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

int main() {
    // 4096 choices of 4 experts (a cluster of CTAs), one matrix of 64 x 64 and its product with itself
    const int n = 4096, E = 4;
    char* d = nullptr;
    if (cudaMalloc(&d, 4 << 20) != cudaSuccess || cudaMemset(d, 0, 4 << 20) != cudaSuccess) return 2;
    int* at = reinterpret_cast<int*>(d);
    pnq_expert_plan plan = {at, at + 8, at + 16, at + 16 + n, at + 16 + 2 * n, n, 1, E};
    const int* ids = at + 16 + 3 * n;
    uint8_t *codes = reinterpret_cast<uint8_t*>(d + (1 << 20)), *scales = codes + 64 * 32;
    float* y = reinterpret_cast<float*>(d + (2 << 20));
    int32_t shape[3];
    for (int round = 0; round < 2; ++round) {
        none_left = round == 0;
        const int a = pnq_expert_sort(ids, &plan, 0);
        const int b = pnq_fp4_gemm(PNQ_NVFP4, codes, scales, 64, codes, scales, 64, 64, 1.0f, PNQ_F32, y, 0, 0);
        const int c = pnq_fp4_gemm_shape(PNQ_NVFP4, 64, 64, 1 << 16, shape, shape + 1, shape + 2);
        none_left = false;
        std::printf("%d %d %d\n", a, b, c);
    }
    return cudaDeviceSynchronize() == cudaSuccess ? 0 : 3;
}
"""


def test_no_exception_leaves_a_c_entry(tmp_path):
    gxx = shutil.which("g++")
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not gxx or not os.path.exists(nvcc):
        pytest.skip("no compiler")
    src, exe, lib = tmp_path / "client.cpp", tmp_path / "client", os.path.dirname(pnq.lib_path())
    src.write_text(CLIENT)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    subprocess.check_call([gxx, "-std=c++17", "-rdynamic", "-I", os.path.join(ROOT, "include"), "-I", os.path.join(cuda, "include"), str(src),
                           "-L", lib, "-lpnq", "-L", os.path.join(cuda, "lib64"), "-lcudart", f"-Wl,-rpath,{lib}",
                           f"-Wl,-rpath,{os.path.join(cuda, 'lib64')}", "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    first, second = ([int(v) for v in line.split()] for line in r.stdout.splitlines())
    assert first == [pnq.Status.ERR_CUDA] * 3 and second == [0] * 3
