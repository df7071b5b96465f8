"""The int8 product's kernels that redistribute registers, where a compiler gave them fewer than they redistribute: those kernels
alone are refused, before a launch, and nothing else is.  The host code runs over a stand-in for the CUDA runtime that says how
many registers a kernel has and writes down what is launched; no test here touches a GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

from quantized_routed_expert_softmax_gb300 import build

RUNTIME = r"""
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime_api.h>
static int regs, launches;
extern "C" {
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
unsigned __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return 0; }
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void*) { *k = nullptr; return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { ++launches; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) { *a = cudaFuncAttributes{}; a->numRegs = regs; return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { ++launches; return cudaSuccess; }
}
namespace moe {
cudaError_t tensor_map(CUtensorMap*, CUtensorMapDataType, CUtensorMapSwizzle, int, const void*, const int64_t*, const int64_t*, const int64_t*) {
    return cudaSuccess;
}
cudaError_t launch_stream_int8(const void*, int64_t, const void*, int64_t, int64_t, int64_t, const int32_t*, int, void*, int, int, cudaStream_t) {
    ++launches;
    return cudaSuccess;
}
cudaError_t configure_int8_codec() { return cudaSuccess; }
cudaError_t configure_int8_kernels();
cudaError_t launch_int8_matmul(const void*, int64_t, const void*, int64_t, int64_t, int64_t, const int32_t*, int, void*, int, int32_t*, int, cudaStream_t);
}
extern "C" int configure(int n) { regs = n; return moe::configure_int8_kernels(); }
// launches of a product of P rows of K columns, or -1 where it is refused
extern "C" int product(int64_t P, int64_t K, int act, int ot) {
    launches = 0;
    static char buf[4096];
    const cudaError_t e = moe::launch_int8_matmul(buf, P, buf, 1, 64, K, nullptr, act, buf, ot, reinterpret_cast<int32_t*>(buf), 152, nullptr);
    return e != cudaSuccess ? (launches ? -2 : -1) : launches;
}
"""


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    try:
        cc = build.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    d = tmp_path_factory.mktemp("registers")
    src, so = d / "runtime.cpp", d / "product.so"
    src.write_text(RUNTIME)
    obj, cxx = d / "int8_gemm.o", shutil.which("g++") or "g++"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")
    subprocess.run([cc, *build.ARCH, *build.FLAGS, "-c", os.path.join(build.CSRC, "int8_gemm.cu"), "-o", str(obj)], check=True, capture_output=True)
    subprocess.run([cxx, "-shared", "-fPIC", "-std=c++17", "-I" + include, str(src), str(obj), "-o", str(so)], check=True, capture_output=True)
    lib = ctypes.CDLL(str(so), mode=os.RTLD_LOCAL | os.RTLD_NOW | getattr(os, "RTLD_DEEPBIND", 0))
    lib.product.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    return lib


@pytest.mark.parametrize("registers", [64, 71, 72, 80])
def test_only_the_kernels_concerned_are_refused(L, registers):
    assert L.configure(registers) == 0
    for act in (0, 1, 2):
        for ot in (0, 1):
            assert L.product(16, 65536, act, ot) == 1 and L.product(500, 1024, act, ot) == 1 and L.product(50, 32, act, ot) == 1
            assert L.product(17, 1056, act, ot) == (1 if registers >= 72 else -1)
