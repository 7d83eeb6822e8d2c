"""Rows beyond 32-bit element and byte offsets: the last rows of a large call equal the same rows in a
small one, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB of device memory")
    yield
    torch.cuda.empty_cache()


def act_context(bep, rows):
    return bep.Context(bep.Config(1, 1, 1, 1, rows, 64, 64, bep.BEP_TRAIN))


def test_activation_past_32_bits(lib):
    bep = lib
    rows, F, last = (1 << 22) + 77, 2048, 300      # 17e9 elements of h, more than 2^30 vectors of 8
    tail = torch.randn(last, 2 * F, device=DEV).bfloat16()
    dtail = torch.randn(last, F, device=DEV).bfloat16()
    small, s_again = torch.empty_like(dtail), torch.empty_like(dtail)
    k = bep.ActCheckpoint(last, F)
    s_dh = torch.empty_like(tail)
    ctx = act_context(bep, last)
    bep.bep_swiglu(ctx, tail, small, k.codes, k.scales)
    bep.bep_swiglu_bwd(ctx, dtail, k.codes, k.scales, s_dh, s_again)
    ctx.close()
    h = torch.zeros(rows, 2 * F, dtype=torch.bfloat16, device=DEV)
    h[-last:] = tail
    a = torch.full((rows, F), 7.0, dtype=torch.bfloat16, device=DEV)
    K = bep.ActCheckpoint(rows, F)
    ctx = act_context(bep, rows)
    bep.bep_swiglu(ctx, h, a, K.codes, K.scales)
    assert bep.bep_status(ctx) == 0
    assert torch.equal(a[-last:], small) and torch.equal(K.codes[-last:], k.codes)
    assert torch.equal(K.scales[-last:], k.scales)
    assert not a[:-last].any().item()
    da = a                                          # its own rows are not needed any more
    da.zero_()
    da[-last:] = dtail
    dh = h
    bep.bep_swiglu_bwd(ctx, da, K.codes, K.scales, dh)
    assert bep.bep_status(ctx) == 0
    assert torch.equal(dh[-last:], s_dh) and not dh[:-last].any().item()
    ctx.close()


def test_4_bit_rows_past_32_bits(lib):
    bep = lib
    T, K, H, Hp, E = 160_000, 8, 7168, 1728, 8      # codes 4.6e9 bytes, y 2.2e9 elements
    rows = T * K
    x = torch.randn(1, T, H, device=DEV).bfloat16()
    w = torch.randn(E, H, Hp, device=DEV).bfloat16()
    ctx = bep.Context(bep.Config(1, E, E, K, T, H, Hp, bep.BEP_TRAIN))
    q = bep.MxWeight(ctx)
    bep.bep_mx_quantize_weight(ctx, w, q.codes, q.scales)
    # expert k takes every token's k-th copy, in token order
    dest = (torch.arange(K, device=DEV) * T + torch.arange(T, device=DEV).unsqueeze(1)).int().view(1, T, K).contiguous()
    cu = torch.full((1, 2 * E + 1), rows, dtype=torch.int32, device=DEV)
    cu[0, :E + 1] = torch.arange(E + 1, device=DEV) * T
    se = torch.full((1, E), -1, dtype=torch.int32, device=DEV)
    r = bep.MxRows(rows, H)
    y = torch.empty(rows, Hp, dtype=torch.bfloat16, device=DEV)
    bep.bep_dispatch_mx(ctx, x, dest, r.codes, r.scales)
    bep.bep_grouped_gemm_mx(ctx, cu, se, r.codes, r.scales, q.codes, q.scales, y)
    assert bep.bep_status(ctx) == 0
    ctx.close()
    last = 500
    ctx = bep.Context(bep.Config(1, E, E, 1, last, H, Hp, bep.BEP_TRAIN))
    one = bep.MxRows(last, H)
    bep.bep_dispatch_mx(ctx, x[:, -last:].contiguous(), torch.arange(last, dtype=torch.int32, device=DEV).view(1, last, 1),
                        one.codes, one.scales)
    for e in (0, E - 1):
        cu = torch.zeros((1, 2 * E + 1), dtype=torch.int32, device=DEV)
        cu[0, e + 1:] = last
        z = torch.empty(last, Hp, dtype=torch.bfloat16, device=DEV)
        bep.bep_grouped_gemm_mx(ctx, cu, se, one.codes, one.scales, q.codes, q.scales, z)
        assert bep.bep_status(ctx) == 0
        end = (e + 1) * T
        assert torch.equal(r.codes[end - last:end], one.codes)
        assert torch.equal(y[end - last:end], z)
    ctx.close()
