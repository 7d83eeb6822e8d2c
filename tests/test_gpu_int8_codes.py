"""Codes of activations that lie close to a tie: the fp32 activation is rounded once, to its integer."""
import numpy as np
import pytest
import torch

import int8_ref as ref
from test_gpu_mx import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("rows,F", [(4096, 1024), (300, 8256), (5000, 192)])
def test_activation_codes_near_ties(lib, rows, F):
    """From a gate of 32 on, the sigmoid is 1 in fp32 and the activation is the product of two bf16 numbers, which fp32
    holds exactly. 127 v / m is then a quotient of integers of 16 bits, and fp64 tells which side of a tie it lies on."""
    bep = lib
    ctx = bep.Context(bep.Config(1, 1, 1, 1, rows, 64, 64, bep.BEP_TRAIN))
    gen = torch.Generator(DEV).manual_seed(rows)
    h = torch.randn(rows, 2 * F, device=DEV, generator=gen)
    h[:, :F] = 32 + 32 * torch.rand(rows, F, device=DEV, generator=gen)
    h = h.bfloat16()
    # ties and their neighbours: m = 127 * 64, v = (k + 1/2) * 64 and v a bf16 step of the gate off it
    h[0, :F] = 64
    h[0, F:] = (torch.arange(F, device=DEV) % 127 + 0.5).bfloat16()
    h[0, F] = 127
    h[0, 1:F:3] = 63.5
    rq = bep.IntRows(rows, F)
    bep.bep_swiglu_int(ctx, h, rq.codes, rq.scales)
    assert bep.bep_status(ctx) == 0
    v = f64(h)
    codes, scales = ref.quantise(v[:, :F] * v[:, F:])
    assert np.array_equal(rq.scales.cpu().numpy(), scales)
    got = rq.codes.cpu().numpy()
    assert np.array_equal(got, codes), int((got != codes).sum())
    ctx.close()
