"""The 8-bit product and the products of any width set their kernels up once a device, not once a context: by stand-ins
for the CUDA runtime and the kernels on the host (CPU)."""
import ctypes
import os
import subprocess

import pytest

import moe_expert_dispatch_online_gb300 as bep
from moe_expert_dispatch_online_gb300 import _build
from test_create_faults import RUNTIME, SHIM, create, number

PARTS = r"""
#include "bep_internal.cuh"
extern "C" { int refused = 0, i8_setups = 0, ragged_setups = 0, i8_pairs = 0, ragged_pairs = 0; }
namespace bep {
cudaError_t plan_setup(int) { return cudaSuccess; }
cudaError_t gemm_setup(int) { return cudaSuccess; }
cudaError_t mx_setup(int, int* clusters) { *clusters = 76; return cudaSuccess; }
cudaError_t i8_setup(int, int* n) { ++i8_setups; *n = 75; return refused ? cudaErrorUnknown : cudaSuccess; }
cudaError_t ragged_setup(int, int* n) { ++ragged_setups; *n = 74; return refused ? cudaErrorUnknown : cudaSuccess; }
cudaError_t launch_grouped_gemm_i8(const Dims&, const Workspace&, const int32_t*, const int32_t*, const int8_t*,
                                   const float*, const int8_t*, const float*, uint16_t*, int clusters, cudaStream_t) {
    i8_pairs = clusters;
    return cudaSuccess;
}
cudaError_t launch_ragged(const Dims&, const Workspace&, const int32_t*, const int32_t*, const uint16_t*, int64_t, int,
                          const uint16_t*, int, int, float, const uint16_t*, int64_t, uint16_t*, int64_t, int, int pairs, cudaStream_t) {
    ragged_pairs = pairs;
    return cudaSuccess;
}
cudaError_t launch_ragged_dw(const Dims&, const Workspace&, const int32_t*, const int32_t*, const uint16_t*, int64_t, int,
                             const uint16_t*, int64_t, int, float, int, float*, int, int pairs, cudaStream_t) {
    ragged_pairs = pairs;
    return cudaSuccess;
}
}
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    d = tmp_path_factory.mktemp("once")
    for name, text in (("shim.h", "#include <atomic>\n" + SHIM), ("runtime.cpp", RUNTIME), ("parts.cpp", PARTS)):
        (d / name).write_text(text)
    so = d / "fake.so"
    subprocess.run([_build.nvcc(), "-x", "c++", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-cudart", "none",
                    *("-Xlinker", "-z", "-Xlinker", "lazy", "-Xlinker", "-Bsymbolic"), "-include", str(d / "shim.h"), "-I", _build.CSRC,
                    "-o", str(so), os.path.join(_build.CSRC, "bep.cu"), str(d / "runtime.cpp"), str(d / "parts.cpp")], check=True)
    lib = ctypes.CDLL(str(so), mode=os.RTLD_LAZY)
    lib.bep_destroy.argtypes = [ctypes.c_void_p]
    lib.bep_destroy.restype = None
    p, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    lib.bep_ragged_gemm.argtypes = [p, p, p, p, i64, i32, p, i32, i32, f32, p, i64, p, i64, p]
    lib.bep_ragged_gemm_dw.argtypes = [p, p, p, p, i64, i32, p, i64, i32, f32, i32, p, p]
    return lib


def calls(lib, h):
    p, q = ctypes.c_void_p(4096), ctypes.c_void_p(8192)
    return (lib.bep_grouped_gemm_int(h, p, p, p, p, p, p, p, None),
            lib.bep_ragged_gemm(h, p, p, p, 64, 64, p, 64, 0, 1.0, None, 0, q, 64, None),
            lib.bep_ragged_gemm_dw(h, p, p, p, 64, 64, p, 64, 64, 1.0, 0, p, None))


def test_once_a_device(fake):
    counts = lambda: tuple(number(fake, n).value for n in ("i8_setups", "ragged_setups"))
    handles = [create(fake, 0) for _ in range(3)]
    assert all(rc == bep.BEP_OK for rc, _ in handles)
    # a set-up that fails is tried again
    number(fake, "refused").value = 1
    assert calls(fake, handles[0][1]) == (bep.BEP_ERR_CUDA,) * 3 and counts() == (1, 2)
    number(fake, "refused").value = 0
    for _, h in handles:
        for _ in range(2):
            assert calls(fake, h) == (bep.BEP_OK,) * 3
            assert counts() == (2, 3)
            assert (number(fake, "i8_pairs").value, number(fake, "ragged_pairs").value) == (75, 74)
        number(fake, "i8_pairs").value = number(fake, "ragged_pairs").value = 0
    for _, h in handles:
        fake.bep_destroy(h)
    assert number(fake, "allocated").value == 0
