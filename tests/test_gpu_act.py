"""The gated activation and its 8-bit checkpoint on the GPU against the 64-bit reference: codes
exactly, activations and gradients within one bf16 rounding of the fp32 result."""
import numpy as np
import pytest
import torch

import experts_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def context(bep, R, S, K):
    return bep.Context(bep.Config(R, R * K, K, K, S, 64, 64, bep.BEP_TRAIN))


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().to(DEV)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def guarded(shape, dtype):
    n = int(np.prod(shape))
    raw = torch.empty(n + 8192, dtype=dtype, device=DEV)
    raw.view(torch.uint8).fill_(0x5A)
    return raw, raw[4096:4096 + n].view(shape)


def intact(raw):
    b = raw.view(torch.uint8)
    e = 4096 * raw.element_size()
    return bool((b[:e] == 0x5A).all() and (b[-e:] == 0x5A).all())


@pytest.mark.parametrize("R,S,K,F", [(1, 1, 1, 32), (1, 1, 3, 64), (2, 64, 2, 64), (3, 41, 3, 480), (1, 7, 1, 8192),
                                     (1, 333, 2, 96), (8, 129, 4, 1024)])
def test_activation_checkpoint_and_gradient(lib, R, S, K, F):
    bep = lib
    rows = R * S * K
    rng = np.random.default_rng([rows, F])
    h = bf16(rng.normal(size=(rows, 2 * F)) * np.exp2(rng.integers(-6, 4, size=(rows, 1))))
    da = bf16(rng.normal(size=(rows, F)))
    ctx = context(bep, R, S, K)
    (ra, a), (rq, q), (rs, s) = (guarded((rows, F), torch.bfloat16), guarded((rows, 2 * F), torch.int8),
                                 guarded((rows, 2 * F // 32), torch.uint8))
    bep.bep_swiglu(ctx, h, a, q, s)
    (rd, dh), (rb, again) = guarded((rows, 2 * F), torch.bfloat16), guarded((rows, F), torch.bfloat16)
    bep.bep_swiglu_bwd(ctx, da, q, s, dh, again)
    assert bep.bep_status(ctx) == 0
    assert all(map(intact, (ra, rq, rs, rd, rb)))
    hd, dd = f64(h), f64(da)
    wq, ws = ref.mx8(hd)
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)
    # bf16 rounding 2^-8, and the fp32 product: 4 roundings, the hardware's exponential (2 units and
    # 2^-23 |g| from the scaled argument) and reciprocal, below 2^-18 for |g| < 32
    tol = 2.0 ** -8 + 2.0 ** -18
    wa = ref.swiglu(hd)
    assert np.all(np.abs(f64(a) - wa) <= tol * np.abs(wa) + 1e-37)
    hv = ref.mx8_values(wq, ws)
    wd, wb = ref.swiglu_bwd(hv, dd), ref.swiglu(hv)
    # dg's bracket s + g s (1 - s) cancels near g = -1.28: its error scales with |da u|
    slack = np.concatenate((np.abs(dd * hv[:, F:]), np.zeros_like(dd)), 1) * 2.0 ** -18
    assert np.all(np.abs(f64(dh) - wd) <= tol * np.abs(wd) + slack + 1e-37)
    assert np.all(np.abs(f64(again) - wb) <= tol * np.abs(wb) + 1e-37)
    # without a checkpoint, and without the activation again
    plain = torch.empty_like(a)
    bep.bep_swiglu(ctx, h, plain)
    dh2 = torch.empty_like(dh)
    bep.bep_swiglu_bwd(ctx, da, q, s, dh2)
    assert torch.equal(plain, a) and torch.equal(dh2, dh)
    ctx.close()


def test_special_values(lib):
    bep = lib
    F = 64
    h = np.zeros((8, 2 * F))
    h[1, 3] = np.inf
    h[2, 70] = np.nan
    h[3] = 3e38
    h[4] = -3e38
    h[5, :32] = 1e-40                      # subnormal in bf16
    h[6, :F] = np.linspace(-200, 200, F)
    h[6, F:] = 1.0
    h[7, 0], h[7, 1] = 254.0, 127.0        # ties in int8: 254 = 127 * 2, 127 / 2 = 63.5 -> 64
    h[7, 2], h[7, 3] = 1.0, 3.0            # 0.5 -> 0, 1.5 -> 2
    ht = bf16(h)
    ctx = context(bep, 1, 8, 1)
    a = torch.empty(8, F, dtype=torch.bfloat16, device=DEV)
    k = bep.ActCheckpoint(8, F)
    bep.bep_swiglu(ctx, ht, a, k.codes, k.scales)
    hd = f64(ht)
    wq, ws = ref.mx8(hd)
    assert np.array_equal(k.codes.cpu().numpy(), wq) and np.array_equal(k.scales.cpu().numpy(), ws)
    assert wq[7, 1] == 64 and wq[7, 2] == 0 and wq[7, 3] == 2 and ws[1, 0] == 255 and ws[2, 2] == 255
    dh = torch.empty(8, 2 * F, dtype=torch.bfloat16, device=DEV)
    bep.bep_swiglu_bwd(ctx, torch.ones_like(a), k.codes, k.scales, dh)
    d = f64(dh)
    assert np.isnan(d[1, :32]).all() and np.isnan(d[1, F:F + 32]).all()      # the block of the infinity
    assert np.isfinite(d[1, 32:F]).all() and np.isfinite(d[1, F + 32:]).all()
    assert np.isnan(d[2, :32]).all() and np.isfinite(d[2, 32:F]).all()       # u's block: dg only
    assert np.isfinite(d[[0, 5, 6, 7]]).all()
    assert np.all(d[0] == 0)
    av = f64(a)
    assert np.isnan(av[2, 6]) and np.isfinite(av[6]).all()
    ctx.close()


def test_another_stream_no_rows_and_refusals(lib):
    bep = lib
    ctx = context(bep, 2, 500, 2)
    rows, F = 2000, 256
    h = torch.randn(rows, 2 * F, device=DEV).bfloat16()
    a, b = torch.empty(rows, F, dtype=torch.bfloat16, device=DEV), torch.empty(rows, F, dtype=torch.bfloat16, device=DEV)
    k = bep.ActCheckpoint(rows, F)
    bep.bep_swiglu(ctx, h, a)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    bep.bep_swiglu(ctx, h, b, stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    for bad, err in ((lambda: bep.bep_swiglu(ctx, h.float(), a), TypeError),
                     (lambda: bep.bep_swiglu(ctx, h[:, ::2], a), ValueError),
                     (lambda: bep.bep_swiglu(ctx, h[:-1], a), ValueError),
                     (lambda: bep.bep_swiglu(ctx, h, a, k.codes, None), bep.BepError),
                     (lambda: bep.bep_swiglu(ctx, h, a, k.codes.view(torch.uint8), k.scales), TypeError),
                     (lambda: bep.bep_swiglu_bwd(ctx, a, k.codes, k.scales, a), ValueError),
                     (lambda: bep.bep_swiglu_bwd(ctx, a, k.codes, None, h), ValueError)):
        with pytest.raises(err):
            bad()
    odd = torch.empty(2000 * 24 * 3 + 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(bep.BepError) as e:     # F = 24 is not a multiple of 32
        bep.bep_swiglu(ctx, odd[:2000 * 48].view(2000, 48), torch.empty(2000, 24, dtype=torch.bfloat16, device=DEV))
    assert e.value.code == bep.BEP_ERR_ARG
    raw = torch.empty(rows * 2 * F + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(bep.BepError) as e:     # 2 bytes off a 16-byte boundary
        bep.bep_swiglu(ctx, raw[1:1 + rows * 2 * F].view(rows, 2 * F), a)
    assert e.value.code == bep.BEP_ERR_ALIGN
    assert bep.bep_status(ctx) == 0
    ctx.close()
    ctx = context(bep, 2, 0, 2)
    bep.bep_swiglu(ctx, h[:0], a[:0])
    assert bep.bep_status(ctx) == 0
    ctx.close()
