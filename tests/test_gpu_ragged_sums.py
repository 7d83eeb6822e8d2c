"""Grouped products of any width and their gradients over long reductions: sums are held in fp32 and each chain of the
tensor core's truncating steps is short, so that the error does not grow with the number of steps."""
import pytest
import torch

from test_gpu_int8 import one_rank

pytestmark = pytest.mark.gpu
DEV = "cuda"

def bound(n, chain):
    """Relative to the sum S of n positive products, `chain` of them until a tensor core's sum is added to one in fp32. A
    step of 16 truncates its chain's sum, S * chain / n at most, by 2^-22 of it: chain / 16 * 2^-22 in all. Each of the
    n / chain additions, and of those of up to 16 parts, rounds by 2^-24 of S. (One chain over all n would lose about half a
    unit of 2^-23 of S / 2 in each of the n / 16 steps at least: 2e-5 at 16,384, and 7.7e-5 as measured.)"""
    return chain / 16 * 2.0 ** -22 + (n / chain + 16) * 2.0 ** -24


def positive(shape, gen):
    return (0.5 + 0.5 * torch.rand(shape, device=DEV, generator=gen)).bfloat16()


def split3(v):
    """fp64 -> three bf16 numbers whose sum is within 2^-24 of it."""
    out = []
    for _ in range(3):
        h = v.bfloat16()
        out.append(h)
        v = v - h.double()
    return torch.stack(out, -1)


# rows of each of two experts, K, N, something to add
@pytest.mark.parametrize("rows,K,N,add", [
    (20, 16384, 16, False),        # parts
    (20, 16384, 40, True),
    (1500, 16384, 104, True),      # two boxes of columns, 8 warps
    (4700, 16384, 104, False),
    (1500, 16384, 1544, False),    # a tile a unit
    (1500, 16384, 1544, True),
    (17000, 16384, 264, False),    # tiles of 256 rows
    (17000, 16384, 136, False),
])
@pytest.mark.parametrize("trans", [False, True])
def test_product_over_a_long_reduction(lib, rows, K, N, add, trans):
    """Positive products whose sum the last step of 16 takes away again: what is left is the error of the sum. Row r is
    a_r b_p with one of four patterns p, column n is c_e d_n, a and d powers of two; the last 12 elements hold -sum b_p c_e
    in three pieces for each pattern."""
    bep = lib
    E, P, n = 2, 4, K - 16
    ctx = bep.Context(bep.Config(1, E, 1, 1, 2 * rows, 64, 64, bep.BEP_INFER))
    cu = torch.tensor([[0, rows, 2 * rows, 2 * rows]], dtype=torch.int32, device=DEV)
    se = torch.full((1, 1), -1, dtype=torch.int32, device=DEV)
    gen = torch.Generator(DEV).manual_seed(K + N)
    b, c = positive((P, n), gen), positive((E, n), gen)
    total = c.double() @ b.double().t()                            # [E, P]
    pieces = split3(total)                                         # [E, P, 3]
    left = (pieces.double().sum(-1) - total).abs().max().item()
    assert left <= 2.0 ** -24 * total.max().item()
    a = torch.exp2(torch.randint(-3, 4, (2 * rows,), device=DEV, generator=gen).float())
    d = torch.exp2(torch.randint(-3, 4, (N,), device=DEV, generator=gen).float())
    pattern = torch.arange(2 * rows, device=DEV) % P
    base = torch.zeros(P, K, dtype=torch.bfloat16, device=DEV)
    base[:, :n] = b
    for p in range(P):
        base[p, n + 3 * p:n + 3 * p + 3] = 1
    x = base[pattern] * a[:, None].bfloat16()
    col = torch.zeros(E, K, dtype=torch.bfloat16, device=DEV)
    col[:, :n] = c
    col[:, n:n + 12] = -pieces.reshape(E, 12)
    w = col[:, None, :] * d[None, :, None].bfloat16() if trans else col[:, :, None] * d[None, None, :].bfloat16()
    y = torch.empty(2 * rows, N, dtype=torch.bfloat16, device=DEV)
    zero = torch.zeros_like(y) if add else None
    bep.bep_ragged_gemm(ctx, cu, se, x, w.contiguous(), y, trans=trans, add=zero)
    assert bep.bep_status(ctx) == 0
    expert = (torch.arange(2 * rows, device=DEV) >= rows).long()
    err = y.double().abs() / (a.double()[:, None] * d.double()[None, :] * total[expert, pattern][:, None])
    # the last step's own truncation, of the whole sum, twice; `left`; y's rounding
    limit = (bound(n, 512) + 2 * 2.0 ** -22 + 2.0 ** -24) * (1 + 2.0 ** -8)
    assert err.max().item() <= limit, (err.max().item(), limit)
    ctx.close()


@pytest.mark.parametrize("rows,K,N", [(16384, 16, 24), (16384, 1096, 200), (16384, 264, 1544), (16384, 2056, 1032)])
def test_gradient_over_many_rows(lib, rows, K, N):
    bep = lib
    ctx, cu, se = one_rank(bep, rows, 64, 64)
    gen = torch.Generator(DEV).manual_seed(K)
    x, dy = positive((rows, K), gen), positive((rows, N), gen)
    g = torch.empty(1, K, N, device=DEV)
    bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g)
    assert bep.bep_status(ctx) == 0
    want = x.double().t() @ dy.double()
    err = ((g[0].double() - want).abs() / want).max().item()
    assert err <= bound(rows, 256), err
    ctx.close()
