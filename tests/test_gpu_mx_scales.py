"""The row scales of the 4-bit product: rewritten between queued calls by other powers of two for every row,
so that one stale scale anywhere would show as a row that is not its own multiple."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("R,S,E,K,H,Hp", [(2, 2000, 4, 2, 2560, 512), (4, 40, 32, 4, 7168, 320), (1, 3000, 2, 1, 192, 1344)])
def test_scales_rewritten_between_calls(lib, R, S, E, K, H, Hp):
    bep = lib
    cfg = bep.Config(R, E, E // R, K, S, H, Hp, bep.BEP_TRAIN)
    ctx = bep.Context(cfg)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(H)
    w = torch.empty(E, H, Hp, device=DEV).normal_(0, 0.05, generator=gen).bfloat16()
    q = bep.MxWeight(ctx)
    bep.bep_mx_quantize_weight(ctx, w, q.codes, q.scales)
    rows = R * S * K
    x = torch.empty(R, S, H, device=DEV).normal_(generator=gen).bfloat16()
    r = bep.MxRows(rows, H)
    r.scales.zero_()
    dest = torch.arange(rows, dtype=torch.int32, device=DEV).view(R, S, K)
    bep.bep_dispatch_mx(ctx, x, dest, r.codes, r.scales)
    cu = torch.full((R, E + cfg.B + 1), cfg.C, dtype=torch.int32, device=DEV)
    cu[:, :E + 1] = (torch.arange(E + 1, device=DEV) * cfg.C // E).int()
    se = torch.full((R, cfg.B), -1, dtype=torch.int32, device=DEV)
    base = r.scales.clone()
    assert int(base[:, :H // 32].min()) > 40 and int(base[:, :H // 32].max()) < 200
    y0 = torch.empty(rows, Hp, dtype=torch.bfloat16, device=DEV)
    bep.bep_grouped_gemm_mx(ctx, cu, se, r.codes, r.scales, q.codes, q.scales, y0)
    assert torch.isfinite(y0).all()
    shifts = [torch.randint(-20, 21, (rows, 1), device=DEV, generator=gen) for _ in range(10)]
    scales = [(base.int() + s).to(torch.uint8) for s in shifts]
    y = [torch.empty_like(y0) for _ in shifts]
    for s, out in zip(scales, y):
        r.scales.copy_(s)
        bep.bep_grouped_gemm_mx(ctx, cu, se, r.codes, r.scales, q.codes, q.scales, out)
    assert bep.bep_status(ctx) == 0
    for s, out in zip(shifts, y):
        # a power of two scales every partial sum and every rounding exactly
        assert torch.equal(out.float(), y0.float() * torch.exp2(s.float()))
    ctx.close()
