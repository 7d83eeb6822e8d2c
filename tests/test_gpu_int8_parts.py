"""The 8-bit product with so few units that the reduction is cut into parts: to the bit."""
import numpy as np
import pytest
import torch

import int8_ref as ref
from kernel_forms import expect
from test_gpu_int8 import bits, weights
from test_gpu_mx import bf16

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rows_of(bep, ctx, n, H, seed):
    rng = np.random.default_rng([n, H, seed])
    x = bf16(rng.normal(size=(1, n, H)))
    r = bep.IntRows(n, H)
    dest = torch.arange(n, dtype=torch.int32, device=DEV).view(1, n, 1)
    bep.bep_dispatch_int(ctx, x, dest, r.codes, r.scales)
    return r


def tables(E, B, lens, slots):
    """lens: (expert, rows) in ascending order of the experts; slots: (expert, rows)."""
    n = np.zeros(E + B, int)
    for e, k in lens:
        n[e] = k
    for j, (_, k) in enumerate(slots):
        n[E + j] = k
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV).view(1, -1)
    se = torch.tensor([[e for e, _ in slots] + [-1] * (B - len(slots))], dtype=torch.int32, device=DEV)
    return cu, se, [*lens, *slots]


# H' of an odd and an even number of tiles of 128, alone and paired; H of two parts and of eight
@pytest.mark.parametrize("H,Hp,lens,slots", [
    (1792, 512, [(1, 1)], []),
    (7168, 512, [(0, 1), (3, 1)], []),
    (7168, 576, [(0, 2)], [(3, 1)]),
    (2752, 384, [(2, 5)], [(2, 3), (77, 2)]),      # a slot whose expert does not exist
    (7168, 2048, [(1, 1), (2, 1)], []),
    (1792, 256, [(0, 33)], []),                    # the second group of epilogue warps has a row
    (7168, 256, [(1, 38)], []),
    (7232, 192, [(0, 30), (3, 8)], []),            # a last stage of half the length
    (7168, 64, [(0, 1), (1, 31), (2, 1), (3, 5)], []),
])
def test_parts(lib, H, Hp, lens, slots):
    bep = lib
    E, B = 4, 3
    n = sum(k for _, k in lens) + sum(k for _, k in slots)
    ctx = bep.Context(bep.Config(1, E, B, 1, n, H, Hp, bep.BEP_INFER))
    w = weights(bep, ctx)
    r = rows_of(bep, ctx, n, H, 1)
    cu, se, runs = tables(E, B, lens, slots)
    q, s = r.codes.cpu().numpy(), r.scales.cpu().numpy()
    wq, ws = w.codes.cpu().numpy(), w.scales.cpu().numpy()
    y = torch.empty(n, Hp, dtype=torch.bfloat16, device=DEV)

    def call():
        bep.bep_grouped_gemm_int(ctx, cu, se, r.codes, r.scales, w.codes, w.scales, y)

    expect(call, "grouped_gemm_i8_kernel<64, true>")
    for _ in range(3):
        y.fill_(9.0)
        call()
        assert bep.bep_status(ctx) == (bep.BEP_DERR_BOUNDS if any(e >= E for e, _ in slots) else 0)
        bep.bep_clear_status(ctx)
        got, at = bits(y), 0
        for e, k in runs:
            if e < E:
                assert np.array_equal(got[at:at + k], ref.product_bits(q[at:at + k], s[at:at + k], wq[e], ws[e])), e
            else:
                assert (y[at:at + k] == 9).all()
            at += k
    ctx.close()


def test_other_numbers_of_parts_in_turn(lib):
    """One context, whose table and so the number of units and of their parts changes from call to call, without a wait."""
    bep = lib
    E, B, n, H, Hp = 6, 1, 8, 7168, 512
    ctx = bep.Context(bep.Config(1, E, B, 1, n, H, Hp, bep.BEP_INFER))
    w = weights(bep, ctx)
    r = rows_of(bep, ctx, n, H, 2)
    splits = [[(0, 8)], [(e, 1) for e in range(5)], [(1, 3), (5, 2)], [], [(4, 1)], [(e, 1) for e in range(6)]]
    t = [tables(E, B, s, []) for s in splits]
    ys = [torch.full((n, Hp), 9.0, dtype=torch.bfloat16, device=DEV) for _ in t]
    for (cu, se, _), y in zip(t, ys):
        bep.bep_grouped_gemm_int(ctx, cu, se, r.codes, r.scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0
    q, s = r.codes.cpu().numpy(), r.scales.cpu().numpy()
    wq, ws = w.codes.cpu().numpy(), w.scales.cpu().numpy()
    for (_, _, runs), y in zip(t, ys):
        got, at = bits(y), 0
        for e, k in runs:
            assert np.array_equal(got[at:at + k], ref.product_bits(q[at:at + k], s[at:at + k], wq[e], ws[e]))
            at += k
        assert (y[at:] == 9).all()
    ctx.close()
