"""The gated activation, its gradient and its 4-bit form where the gate's sigmoid is as small as fp32 holds, or
smaller, and the other factor is large: against the 64-bit reference."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from test_gpu_act import bf16, context, f64

pytestmark = pytest.mark.gpu

# 2^-8 for bf16's rounding; hardware exponential and reciprocal, and the argument's rounding at |g| <= 172,
# 2^-21 + 172 * 2^-23 and a few products: below 2^-15
TOL = 2.0 ** -8 + 2.0 ** -15
TINY = 2.0 ** -126                     # results below are subnormal in bf16 and fp32

GATES = np.r_[-np.arange(80, 96, 0.5), -np.arange(96, 172, 4.0), np.arange(80, 104, 4.0), 0.0, -1.25, 1.0, -40.0]


@pytest.mark.parametrize("up", (1.0, -2.0 ** 40, 2.0 ** 127, 3e38))
def test_tiny_sigmoids(lib, up):
    bep = lib
    rows, F = len(GATES), 64
    h = np.zeros((rows, 2 * F))
    h[:, :F] = GATES[:, None]
    h[:, F:] = up * (1 + np.arange(F) % 32)[::-1] / 32
    ht = bf16(h)
    hd = f64(ht)
    ctx = context(bep, 1, rows, 1)
    a, again = torch.empty(rows, F, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, F, dtype=torch.bfloat16, device="cuda")
    dh = torch.empty(rows, 2 * F, dtype=torch.bfloat16, device="cuda")
    k = bep.ActCheckpoint(rows, F)
    bep.bep_swiglu(ctx, ht, a, k.codes, k.scales)
    da = bf16(np.resize([0.5, -0.75, 2.0 ** -20, 1.0], (rows, F)))
    bep.bep_swiglu_bwd(ctx, da, k.codes, k.scales, dh, again)
    assert bep.bep_status(ctx) == 0
    hv = ref.mx8_values(*ref.mx8(hd))
    big = 3.3895e38                    # bf16's largest: beyond it both sides are infinite
    with np.errstate(over="ignore"):
        for got, want, slack in ((a, ref.swiglu(hd), 0.0), (again, ref.swiglu(hv), 0.0),
                                 # dg's bracket 1 + g (1 - s) cancels near g = -1.28
                                 (dh, ref.swiglu_bwd(hv, f64(da)), 2.0 ** -18)):
            got = f64(got)
            tol = TOL * np.abs(want) + TINY
            if slack:
                s = 1 / (1 + np.exp(-hv[:, :F]))
                tol[:, :F] += slack * np.abs(f64(da) * hv[:, F:]) * s
            over = np.abs(want) > big * (1 - 2.0 ** -8)
            assert np.all((np.abs(got - want) <= tol) | over)
            assert np.all(np.sign(got[over]) == np.sign(want[over]))
    ctx.close()


def test_tiny_sigmoids_in_4_bits(lib):
    bep = lib
    gates = np.r_[-np.arange(84, 90, 0.5), -100.0, -130.0]
    ups = np.array([1.0, 2.0 ** 60, 2.0 ** 120])
    rows, F = len(gates) * len(ups), 64
    h = np.zeros((rows, 2 * F))
    h[:, :F] = np.repeat(gates, len(ups))[:, None]
    h[:, F:] = np.tile(ups, len(gates))[:, None] * np.resize([1.0, -0.375, 0.25, 0.0], F)
    ht = bf16(h)
    ctx = context(bep, 1, rows, 1)
    q = bep.MxRows(rows, F)
    bep.bep_swiglu_mx(ctx, ht, q.codes, q.scales)
    assert bep.bep_status(ctx) == 0
    a = ref.swiglu(f64(ht))
    amax = np.abs(a).max(1)
    seen = amax > 2.0 ** -120          # the format's own scales end at 2^-127
    assert seen.sum() > rows // 2
    wc, wb = ref.mx4(a)
    got, sc = ref.unpack4(q.codes.cpu().numpy()), q.scales.cpu().numpy()[:, :F // 32]
    # ratios 1, 3/8, 1/4 of the largest: not near a rounding boundary unless the largest is
    b = a.reshape(rows, -1, 32)
    frac = np.log2(np.abs(b).max(-1) / 6.0) % 1.0
    v = np.abs(np.ldexp(b, -(wb[..., None].astype(np.int64) - 127)))
    mids = (ref.E2M1[1:] + ref.E2M1[:-1]) / 2
    near = (np.abs(v[..., None] - mids) < 2.0 ** -15 * mids).any((-1, -2)) | (np.minimum(frac, 1 - frac) < 1e-4)
    sure = seen[:, None] & ~near
    assert sure.sum() > rows // 2
    assert np.array_equal(sc[sure], wb[sure])
    assert np.array_equal(got.reshape(rows, -1, 32)[sure], wc.reshape(rows, -1, 32)[sure])
    ctx.close()
