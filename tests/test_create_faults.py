"""bep_create where a part of its set-up fails, by fakes of the failing calls on the host (CPU): bep.cu, which
holds no kernel, is compiled alone as C++ and linked with stand-ins for the CUDA runtime and the other
translation units."""
import ctypes
import os
import subprocess

import pytest

import moe_expert_dispatch_online_gb300 as bep
from moe_expert_dispatch_online_gb300 import _build

# what the shared header's device functions need to pass as C++
SHIM = r"""
#include <cuda_runtime.h>
#undef __device__
#undef __forceinline__
#define __device__
#define __forceinline__ inline
inline void atomicOr(int*, int) {}
inline unsigned __umulhi(unsigned, unsigned) { return 0; }
"""

# the runtime's calls succeed without a device
RUNTIME = r"""
#include <stdlib.h>
#include <cuda_runtime_api.h>
extern "C" {
int allocated = 0;
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t n) { *p = malloc(n); ++allocated; return cudaSuccess; }
cudaError_t cudaFree(void* p) { free(p); --allocated; return cudaSuccess; }
cudaError_t cudaMemset(void*, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
}
"""

# `refused` names the set-up that fails: 1 plan, 2 gemm, 3 the 4-bit product
PARTS = r"""
#include "bep_internal.cuh"
extern "C" { int refused = 0, launches = 0; }
namespace bep {
cudaError_t plan_setup(int) { return refused == 1 ? cudaErrorUnknown : cudaSuccess; }
cudaError_t gemm_setup(int) { return refused == 2 ? cudaErrorUnknown : cudaSuccess; }
cudaError_t mx_setup(int, int* clusters) {
    *clusters = 76;
    return refused == 3 ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t launch_dispatch(const Dims&, const Workspace&, const uint16_t*, const int32_t*, uint16_t*, int, cudaStream_t) {
    ++launches;
    return cudaSuccess;
}
cudaError_t launch_grouped_gemm_mx(const Dims&, const Workspace&, const int32_t*, const int32_t*, const uint8_t*,
                                   const uint8_t*, const uint8_t*, const uint8_t*, uint16_t*, int clusters, cudaStream_t) {
    launches += clusters;
    return cudaSuccess;
}
}
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    d = tmp_path_factory.mktemp("create")
    for name, text in (("shim.h", SHIM), ("runtime.cpp", RUNTIME), ("parts.cpp", PARTS)):
        (d / name).write_text(text)
    so = d / "fake.so"
    # what no test calls stays unresolved; the stand-ins come before a runtime that the process has loaded
    subprocess.run([_build.nvcc(), "-x", "c++", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-cudart", "none",
                    *("-Xlinker", "-z", "-Xlinker", "lazy", "-Xlinker", "-Bsymbolic"), "-include", str(d / "shim.h"), "-I", _build.CSRC,
                    "-o", str(so), os.path.join(_build.CSRC, "bep.cu"), str(d / "runtime.cpp"),
                    str(d / "parts.cpp")], check=True)
    lib = ctypes.CDLL(str(so), mode=os.RTLD_LAZY)
    lib.bep_destroy.argtypes = [ctypes.c_void_p]
    lib.bep_destroy.restype = None
    return lib


def number(lib, name):
    return ctypes.c_int.in_dll(lib, name)


def create(lib, refused):
    number(lib, "refused").value = refused
    c = bep._Config(2, 8, 4, 2, 16, 128, 64, bep.BEP_TRAIN)
    h = ctypes.c_void_p()
    return lib.bep_create(ctypes.byref(c), ctypes.byref(h)), h


def calls(lib, h):
    p = ctypes.c_void_p(4096)
    n0 = number(lib, "launches").value
    rc = lib.bep_dispatch(h, p, p, p, None), lib.bep_grouped_gemm_mx(h, p, p, p, p, p, p, p, None)
    return rc, number(lib, "launches").value - n0


def test_everything_set_up(fake):
    rc, h = create(fake, 0)
    assert rc == bep.BEP_OK
    assert calls(fake, h) == ((bep.BEP_OK, bep.BEP_OK), 1 + 76)
    fake.bep_destroy(h)
    assert number(fake, "allocated").value == 0


@pytest.mark.parametrize("refused", (1, 2))
def test_what_every_context_needs(fake, refused):
    rc, h = create(fake, refused)
    assert rc == bep.BEP_ERR_CUDA and not h.value
    assert number(fake, "allocated").value == 0


def test_the_4_bit_product_alone_is_refused(fake):
    rc, h = create(fake, 3)
    assert rc == bep.BEP_OK
    assert calls(fake, h) == ((bep.BEP_OK, bep.BEP_ERR_CUDA), 1)
    fake.bep_destroy(h)
    assert number(fake, "allocated").value == 0
