"""The 4-bit product behind kernels that are not the library's: whatever writes the segment table, the
rows or their scales just before a product, also a kernel that lets its dependents start before it has
written anything, is waited for."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"

# One CTA: lets its dependents start, sleeps for 0.2 to 0.4 ms, and only then copies n words.
SOURCE = r"""
#include <cuda_runtime.h>
__global__ void late_copy(int* dst, const int* src, long long n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = 0; i < 20; ++i) __nanosleep(10000);
    for (long long i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}
extern "C" int launch_late_copy(int* dst, const int* src, long long n, void* stream) {
    late_copy<<<1, 1024, 0, static_cast<cudaStream_t>(stream)>>>(dst, src, n);
    return static_cast<int>(cudaGetLastError());
}
"""


@pytest.fixture(scope="module")
def late_copy(tmp_path_factory):
    from moe_expert_dispatch_online_gb300 import _build
    d = tmp_path_factory.mktemp("late_copy")
    (d / "late_copy.cu").write_text(SOURCE)
    so = d / "late_copy.so"
    subprocess.run([_build.nvcc(), *_build.ARCH, "-O3", "-Xcompiler", "-fPIC", "-shared", "-o", str(so),
                    str(d / "late_copy.cu")], check=True)
    fn = ctypes.CDLL(str(so)).launch_late_copy
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_void_p]

    def copy(dst, src):
        nbytes = dst.numel() * dst.element_size()
        assert nbytes == src.numel() * src.element_size() and nbytes % 4 == 0
        assert fn(dst.data_ptr(), src.data_ptr(), nbytes // 4, torch.cuda.current_stream().cuda_stream) == 0

    return copy


def tables(R, E, B, C, seed):
    """A segment table that covers every rank's C rows, without slots."""
    rng = np.random.default_rng(seed)
    cu = np.full((R, E + B + 1), C, np.int32)
    cu[:, 0] = 0
    cu[:, 1:E] = np.sort(rng.integers(0, C + 1, size=(R, E - 1)), axis=1)
    return torch.from_numpy(cu).to(DEV)


@pytest.mark.parametrize("last", ("table", "codes", "scales"))
@pytest.mark.parametrize("early", (True, False))
def test_the_kernel_before_is_waited_for(lib, late_copy, last, early):
    bep = lib
    R, S, E, K, H, Hp = 2, 150, 8, 2, 576, 320
    cfg = bep.Config(R, E, E // R, K, S, H, Hp, bep.BEP_TRAIN)
    ctx = bep.Context(cfg)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    w = torch.empty(E, H, Hp, device=DEV).normal_(0, 0.05, generator=gen).bfloat16()
    q = bep.MxWeight(ctx)
    bep.bep_mx_quantize_weight(ctx, w, q.codes, q.scales)
    dest = torch.arange(R * S * K, dtype=torch.int32, device=DEV).view(R, S, K)
    se = torch.full((R, cfg.B), -1, dtype=torch.int32, device=DEV)
    kept = []
    for i in range(2):
        rows = bep.MxRows(R * S * K, H)
        x = torch.empty(R, S, H, device=DEV).normal_(0, 4.0 ** i, generator=gen).bfloat16()
        rows.scales.zero_()
        bep.bep_dispatch_mx(ctx, x, dest, rows.codes, rows.scales)
        kept.append(dict(table=tables(R, E, cfg.B, cfg.C, i), codes=rows.codes, scales=rows.scales))

    def product(t, y):
        bep.bep_grouped_gemm_mx(ctx, t["table"], se, t["codes"], t["scales"], q.codes, q.scales, y)

    want = [torch.empty(R * S * K, Hp, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for t, y in zip(kept, want):
        torch.cuda.synchronize()
        product(t, y)
    torch.cuda.synchronize()
    assert not torch.equal(*want)
    used = {k: v.clone() for k, v in kept[1].items()}
    order = [k for k in used if k != last] + [last]
    got = [torch.empty_like(want[0]) for _ in range(8)]
    for i, y in enumerate(got):
        for k in order:
            late_copy(used[k], kept[i % 2][k]) if early else used[k].copy_(kept[i % 2][k])
        product(used, y)
    assert bep.bep_status(ctx) == 0
    for i, y in enumerate(got):
        assert torch.equal(y.view(torch.int16), want[i % 2].view(torch.int16)), i
    ctx.close()
