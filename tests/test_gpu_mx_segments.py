"""The 4-bit product's work list over more segments than its one block takes at a time (4,096)."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from test_gpu_mx import DEV, bf16, check_product, f64, planned, row_experts, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,S,E,K,B,skew", [(16, 40, 256, 4, None, 1.0), (16, 300, 512, 2, 3, 1.5), (64, 6, 2048, 8, None, 0.5)])
def test_many_segments(lib, R, S, E, K, B, skew):
    bep = lib
    H, Hp = 64, 64
    ctx, t = planned(bep, R, S, E, K, H, Hp, B, seed=7, skew=skew)
    c = ctx.cfg
    assert R * (E + c.B) > 4096
    _, w = weights(bep, ctx)
    x = bf16(np.random.default_rng(R).normal(size=(R, S, H)))
    rows = bep.MxRows(R * S * K, H)
    bep.bep_dispatch_mx(ctx, x, t["dest"], rows.codes, rows.scales)
    raw = torch.full((R * S * K * Hp + 8192,), 9.0, dtype=torch.bfloat16, device=DEV)
    y = raw[4096:4096 + R * S * K * Hp].view(R * S * K, Hp)
    bep.bep_grouped_gemm_mx(ctx, t["cu"], t["se"], rows.codes, rows.scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0
    assert (raw[:4096] == 9).all() and (raw[-4096:] == 9).all()
    xv = ref.mx4_values(ref.unpack4(rows.codes.cpu().numpy()), rows.scales.cpu().numpy()[:, :H // 32])
    wv = ref.mx4_values(ref.unpack4(w.codes.cpu().numpy()),
                        ref.unblock_scales(w.scales.cpu().numpy(), Hp, H // 32))
    expert = row_experts(c, t)
    assert (expert >= 0).all()
    check_product(f64(y), xv, wv, expert, H)
    # one bad entry anywhere refuses the table as a whole
    for u, r in ((0, 3), (R - 1, E)):
        cu = t["cu"].clone()
        cu[u, r] = c.C + 1
        raw.fill_(9.0)
        bep.bep_grouped_gemm_mx(ctx, cu, t["se"], rows.codes, rows.scales, w.codes, w.scales, y)
        assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS and (raw == 9).all()
        bep.bep_clear_status(ctx)
    ctx.close()
