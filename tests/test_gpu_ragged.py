"""Grouped products of any width on the GPU. Most inputs are small integers, whose sums are exact in fp32 in any
order: the outputs have to equal the formula's to the bit. Others are held to fp32 accumulation."""
import numpy as np
import pytest
import torch

import int8_ref as ref
from test_gpu_int8 import bits, one_rank
from test_gpu_mx import f64, planned, row_experts

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(shape, seed, top=4):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device=DEV).bfloat16()


def wide(t, left, right, fill=float("nan")):
    """t [rows, n] as a slice of columns of a wider buffer that holds `fill` elsewhere: (slice, buffer)."""
    buf = torch.full((t.shape[0], left + t.shape[1] + right), fill, dtype=t.dtype, device=t.device)
    buf[:, left:left + t.shape[1]] = t
    return buf[:, left:left + t.shape[1]], buf


def table(lens, R=1, spare=0, slots=()):
    """One rank's table of home segments of the given lengths and of slots (expert, length); rows in total."""
    E = len(lens)
    n = [0] + list(lens) + [length for _, length in slots]
    cu = torch.tensor(np.cumsum(n), dtype=torch.int32, device=DEV).view(1, -1)
    se = torch.tensor([[e for e, _ in slots]], dtype=torch.int32, device=DEV)
    return cu, se, int(sum(n)) + spare


def context(bep, E, B, rows):
    return bep.Context(bep.Config(1, E, B, 1, rows, 64, 64, bep.BEP_TRAIN if B == E else bep.BEP_INFER))


def want_y(x, w, expert, alpha, add, trans):
    w = f64(w)
    y = np.zeros((x.shape[0], w.shape[1] if trans else w.shape[2]))
    for e in np.unique(expert[expert >= 0]):
        at = expert == e
        y[at] = alpha * (f64(x)[at] @ (w[e].T if trans else w[e]))
    return y if add is None else y + f64(add)


def want_g(x, dy, expert, E, alpha):
    g = np.zeros((E, x.shape[1], dy.shape[1]))
    for e in np.unique(expert[expert >= 0]):
        at = expert == e
        g[e] = alpha * (f64(x)[at].T @ f64(dy)[at])
    return g


# R, S, E, top-K, K, N, B (None: training), skew
SHAPES = [
    (1, 1, 2, 1, 8, 8, None, 0.0),
    (1, 1, 8, 3, 7168, 16, 1, 0.0),
    (2, 1, 16, 4, 16, 2048, None, 0.5),
    (2, 37, 8, 2, 72, 40, None, 1.2),
    (1, 300, 2, 1, 520, 136, 1, 0.0),
    (3, 70, 12, 5, 1088, 576, None, 1.0),
    (4, 100, 16, 3, 328, 1000, 2, 1.5),
    (8, 17, 24, 6, 4160, 264, 1, 1.5),
    (2, 500, 6, 2, 24, 1544, None, 0.3),
    (2, 700, 4, 2, 1096, 24, None, 0.6),
    (1, 129, 1, 1, 64, 2048, None, 0.0),
    (2, 900, 2, 1, 64, 8, None, 0.0),
    (1, 1300, 2, 1, 520, 264, None, 0.3),
    (2, 1500, 4, 2, 1096, 200, None, 1.5),
    (3, 2000, 6, 2, 488, 776, 1, 2.0),
]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("R,S,E,top,K,N,B,skew", SHAPES)
def test_product(lib, R, S, E, top, K, N, B, skew, trans):
    bep = lib
    ctx, t = planned(bep, R, S, E, top, 64, 64, B, seed=3, skew=skew)
    expert = row_experts(ctx.cfg, t)
    rows = R * S * top
    x, xb = wide(ints((rows, K), 1), 16, 8)
    w = ints((E, N, K) if trans else (E, K, N), 2)
    add, _ = wide(ints((rows, N), 3, 100), 8, 24)
    y, yb = wide(torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV), 24, 16, 9.0)
    for a, alpha in ((None, 1.0), (add, -0.5)):
        bep.bep_ragged_gemm(ctx, t["cu"], t["se"], x, w, y, trans=trans, alpha=alpha, add=a)
        assert bep.bep_status(ctx) == 0
        want = ref.bf16_bits(want_y(x, w, expert, alpha, a, trans).astype(np.float32))
        assert np.array_equal(bits(y.contiguous()), want)
        assert (yb[:, :24] == 9).all() and (yb[:, 24 + N:] == 9).all()
    ctx.close()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("R,S,E,top,K,N,B,skew", SHAPES)
def test_gradient(lib, R, S, E, top, K, N, B, skew, accumulate):
    bep = lib
    ctx, t = planned(bep, R, S, E, top, 64, 64, B, seed=3, skew=skew)
    expert = row_experts(ctx.cfg, t)
    rows = R * S * top
    x, _ = wide(ints((rows, K), 1), 16, 8)
    dy, _ = wide(ints((rows, N), 2), 8, 8)
    raw = torch.full((E * K * N + 2048,), 3.0, device=DEV)
    g = raw[1024:1024 + E * K * N].view(E, K, N)
    bep.bep_ragged_gemm_dw(ctx, t["cu"], t["se"], x, dy, g, alpha=0.5, accumulate=accumulate)
    assert bep.bep_status(ctx) == 0
    want = want_g(x, dy, expert, E, 0.5) + (3.0 if accumulate else 0.0)
    assert np.array_equal(g.cpu().numpy(), want)
    assert (raw[:1024] == 3).all() and (raw[-1024:] == 3).all()
    ctx.close()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("R,S,E,top,K,N,skew", [
    (2, 2100, 8, 1, 1024, 1040, 0.5),    # an even number of tiles on either side
    (3, 1600, 9, 1, 840, 1096, 2.5),     # an odd one, experts of very different lengths
    (2, 2650, 20, 2, 360, 1000, 0.7),    # three tiles
    (2, 2650, 20, 2, 136, 2048, 0.0),    # dy on the side that is cut into pairs of tiles
])
def test_gradient_of_long_experts(lib, R, S, E, top, K, N, skew, accumulate):
    """Lengths and widths at which two blocks share an operand. The rows behind each segment are another's."""
    bep = lib
    ctx, t = planned(bep, R, S, E, top, 64, 64, seed=4, skew=skew)
    expert = row_experts(ctx.cfg, t)
    rows = R * S * top
    x, _ = wide(ints((rows, K), 1), 8, 16)
    dy, _ = wide(ints((rows, N), 2), 24, 8)
    want = want_g(x, dy, expert, E, 0.5) + (3.0 if accumulate else 0.0)
    for _ in range(2):
        g = torch.full((E, K, N), 3.0, device=DEV)
        bep.bep_ragged_gemm_dw(ctx, t["cu"], t["se"], x, dy, g, alpha=0.5, accumulate=accumulate)
        assert bep.bep_status(ctx) == 0
        assert np.array_equal(g.cpu().numpy(), want)
    ctx.close()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("R,S,E,top,K,N,skew", [
    (2, 1100, 4, 1, 520, 1096, 0.5),     # an odd number of tiles of columns
    (1, 1664, 3, 1, 1544, 264, 2.0),     # two; experts of very different lengths
    (3, 1400, 9, 2, 512, 2048, 0.0),     # nothing ragged but the rows
])
def test_products_of_long_experts(lib, R, S, E, top, K, N, skew, trans):
    """Lengths and widths at which two blocks share the rows."""
    bep = lib
    ctx, t = planned(bep, R, S, E, top, 64, 64, seed=6, skew=skew)
    expert = row_experts(ctx.cfg, t)
    rows = R * S * top
    x, _ = wide(ints((rows, K), 1), 8, 16)
    w = ints((E, N, K) if trans else (E, K, N), 2)
    y, yb = wide(torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV), 24, 16, 9.0)
    want = ref.bf16_bits(want_y(x, w, expert, 0.25, None, trans).astype(np.float32))
    for _ in range(2):
        y.zero_()
        bep.bep_ragged_gemm(ctx, t["cu"], t["se"], x, w, y, trans=trans, alpha=0.25)
        assert bep.bep_status(ctx) == 0
        assert np.array_equal(bits(y.contiguous()), want)
        assert (yb[:, :24] == 9).all() and (yb[:, 24 + N:] == 9).all()
    ctx.close()


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 100, 127, 128, 129, 191, 200, 257, 300])
@pytest.mark.parametrize("K,N", [(104, 72), (72, 104)])
def test_every_segment_height(lib, rows, K, N):
    """The rows behind a segment hold NaN: they reach neither its outputs nor its gradient."""
    bep = lib
    cu, se, n = table([rows, 0, 5], spare=70)
    ctx = bep.Context(bep.Config(1, 3, 1, 1, n, 64, 64, bep.BEP_INFER))
    cu = torch.cat((cu, cu[:, -1:]), 1).contiguous()
    se = torch.full((1, 1), -1, dtype=torch.int32, device=DEV)
    x, dy = ints((n, K), 5), ints((n, N), 6)
    x[rows + 5:], dy[rows + 5:] = float("nan"), float("nan")
    w = ints((3, K, N), 7)
    y = torch.full((n, N), 9.0, dtype=torch.bfloat16, device=DEV)
    bep.bep_ragged_gemm(ctx, cu, se, x, w, y)
    expert = np.full(n, -1)
    expert[:rows], expert[rows:rows + 5] = 0, 2
    want = want_y(torch.nan_to_num(x), w, expert, 1.0, None, False)
    assert np.array_equal(f64(y)[:rows + 5], want[:rows + 5].astype(np.float32).astype(np.float64)) or \
        np.array_equal(bits(y)[:rows + 5], ref.bf16_bits(want[:rows + 5].astype(np.float32)))
    assert (y[rows + 5:] == 9).all()
    # a NaN in the segment behind stays there
    x[rows], dy[rows + 1] = float("nan"), float("nan")
    g = torch.full((3, K, N), 7.0, device=DEV)
    bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g)
    assert bep.bep_status(ctx) == 0
    assert np.array_equal(g[0].cpu().numpy(), f64(x)[:rows].T @ f64(dy)[:rows])
    assert (g[1] == 0).all() and g[2].isnan().all()
    ctx.close()


def test_many_segments_of_one_expert(lib):
    """An expert's rows in its home row on every rank (overflow) and in several slots of one rank."""
    bep = lib
    R, E, B, S, K, N = 4, 8, 1, 300, 136, 24
    ctx = bep.Context(bep.Config(R, E, B, 1, S, 64, 64, bep.BEP_INFER))
    rng = np.random.default_rng(3)
    cu = np.zeros((R, E + B + 1), np.int32)
    for u in range(R):
        cu[u, 1:] = np.sort(rng.integers(0, S + 1, size=E + B))
    se = np.array([[2], [2], [5], [2]], np.int32)
    expert = np.full(R * S, -1)
    for u in range(R):
        for rho in range(E + B):
            expert[u * S + cu[u, rho]:u * S + cu[u, rho + 1]] = rho if rho < E else se[u, rho - E]
    t = torch.from_numpy(cu).to(DEV), torch.from_numpy(se).to(DEV)
    x, dy, w = ints((R * S, K), 1), ints((R * S, N), 2), ints((E, K, N), 3)
    g = torch.empty(E, K, N, device=DEV)
    y = torch.full((R * S, N), 9.0, dtype=torch.bfloat16, device=DEV)
    bep.bep_ragged_gemm_dw(ctx, *t, x, dy, g)
    bep.bep_ragged_gemm(ctx, *t, x, w, y)
    assert bep.bep_status(ctx) == 0
    assert np.array_equal(g.cpu().numpy(), want_g(x, dy, expert, E, 1.0))
    at = expert >= 0
    assert np.array_equal(bits(y)[at], ref.bf16_bits(want_y(x, w, expert, 1.0, None, False).astype(np.float32))[at])
    assert (y.cpu()[torch.from_numpy(~at)] == 9).all()
    ctx.close()


def test_slots_of_one_rank_that_hold_the_same_expert(lib):
    bep = lib
    E, K, N = 4, 40, 56
    cu, se, n = table([3, 0, 17, 0], slots=[(2, 9), (1, 0), (2, 20), (0, 5)])
    ctx = context(bep, E, E, n)
    expert = np.concatenate([np.full(c, e) for e, c in ((0, 3), (2, 17), (2, 9), (2, 20), (0, 5))])
    x, dy = ints((n, K), 1), ints((n, N), 2)
    g = torch.empty(E, K, N, device=DEV)
    bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g)
    assert bep.bep_status(ctx) == 0
    assert np.array_equal(g.cpu().numpy(), want_g(x, dy, expert, E, 1.0))
    ctx.close()


def test_many_slots(lib):
    """More slots than a CTA has threads."""
    bep = lib
    E, K, N = 2048, 8, 16
    rng = np.random.default_rng(1)
    lens, slots = rng.integers(0, 3, size=E), [(int(e), int(n)) for e, n in zip(rng.integers(0, 40, size=E), rng.integers(0, 3, size=E))]
    cu, se, n = table(lens, slots=slots)
    ctx = context(bep, E, E, n)
    expert = np.concatenate((np.repeat(np.arange(E), lens), np.repeat([e for e, _ in slots], [c for _, c in slots])))
    x, dy, w = ints((n, K), 1), ints((n, N), 2), ints((E, K, N), 4)
    g = torch.empty(E, K, N, device=DEV)
    y = torch.empty(n, N, dtype=torch.bfloat16, device=DEV)
    bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g)
    bep.bep_ragged_gemm(ctx, cu, se, x, w, y)
    assert bep.bep_status(ctx) == 0
    assert np.array_equal(g.cpu().numpy(), want_g(x, dy, expert, E, 1.0))
    assert np.array_equal(bits(y), ref.bf16_bits(want_y(x, w, expert, 1.0, None, False).astype(np.float32)))
    ctx.close()


def test_bad_tables(lib):
    bep = lib
    K, N = 40, 24
    cu, se, n = table([3, 4], slots=[(1, 5), (7, 6)], spare=3)   # expert 7 does not exist
    ctx = context(bep, 2, 2, n)
    x, dy, w = ints((n, K), 1), ints((n, N), 2), ints((2, K, N), 3)
    y = torch.full((n, N), 9.0, dtype=torch.bfloat16, device=DEV)
    g = torch.full((2, K, N), 9.0, device=DEV)
    expert = np.array([0] * 3 + [1] * 9 + [-1] * 9)
    bep.bep_ragged_gemm(ctx, cu, se, x, w, y)
    assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
    bep.bep_clear_status(ctx)
    assert (y[12:] == 9).all()
    assert np.array_equal(bits(y)[:12], ref.bf16_bits(want_y(x, w, expert, 1.0, None, False).astype(np.float32))[:12])
    bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g)
    assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
    bep.bep_clear_status(ctx)
    assert np.array_equal(g.cpu().numpy(), want_g(x, dy, expert, 2, 1.0))
    for bad in ([0, 3, 2, 12, 18], [0, 3, 7, 12, n + 1], [-1, 3, 7, 12, 18]):
        cu[0] = torch.tensor(bad, dtype=torch.int32)
        y.fill_(9.0)
        g.fill_(9.0)
        bep.bep_ragged_gemm(ctx, cu, se, x, w, y)
        assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
        bep.bep_clear_status(ctx)
        bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g)
        assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
        bep.bep_clear_status(ctx)
        assert (y == 9).all() and (g == 9).all()
    cu.zero_()   # nobody has rows
    bep.bep_ragged_gemm(ctx, cu, se, x, w, y)
    bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g, accumulate=True)
    assert bep.bep_status(ctx) == 0 and (y == 9).all() and (g == 9).all()
    bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g)
    assert bep.bep_status(ctx) == 0 and (g == 0).all()
    ctx.close()


@pytest.mark.parametrize("R,S,E,top,K,N", [(2, 300, 8, 2, 1096, 200), (1, 4, 8, 2, 5000, 48), (2, 2000, 2, 1, 48, 8)])
def test_real_values(lib, R, S, E, top, K, N):
    """fp32 accumulation: each of the n / 16 steps of a sum truncates it to 2^-22 of the magnitudes at most (as the
    products of 4-bit values), then one bf16 rounding of the rows' outputs. The same call gives the same bits."""
    bep = lib
    ctx, t = planned(bep, R, S, E, top, 64, 64, seed=5, skew=0.5)
    expert = row_experts(ctx.cfg, t)
    rows = R * S * top
    gen = torch.Generator(DEV).manual_seed(1)
    x = torch.randn(rows, K, device=DEV, generator=gen).bfloat16()
    dy = torch.randn(rows, N, device=DEV, generator=gen).bfloat16()
    w = torch.randn(E, K, N, device=DEV, generator=gen).bfloat16()
    add = torch.randn(rows, N, device=DEV, generator=gen).bfloat16()
    y = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
    g = torch.empty(E, K, N, device=DEV)
    bep.bep_ragged_gemm(ctx, t["cu"], t["se"], x, w, y, alpha=0.3, add=add)
    bep.bep_ragged_gemm_dw(ctx, t["cu"], t["se"], x, dy, g, alpha=0.3)
    a = float(np.float32(0.3))
    want = want_y(x, w, expert, a, add, False)
    mag = want_y(x.abs(), w.abs(), expert, a, add.abs(), False)
    assert np.all(np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + (K / 16 + 2) * 2.0 ** -22 * mag)
    want, mag = want_g(x, dy, expert, E, a), want_g(x.abs(), dy.abs(), expert, E, a)
    count = np.bincount(expert, minlength=E)[:, None, None]
    assert np.all(np.abs(g.cpu().numpy() - want) <= (count / 16 + R + 2) * 2.0 ** -22 * mag)
    for _ in range(3):
        y2, g2 = torch.empty_like(y), torch.empty_like(g)
        bep.bep_ragged_gemm(ctx, t["cu"], t["se"], x, w, y2, alpha=0.3, add=add)
        bep.bep_ragged_gemm_dw(ctx, t["cu"], t["se"], x, dy, g2, alpha=0.3)
        assert torch.equal(y2.view(torch.int16), y.view(torch.int16)) and torch.equal(g2, g)
    ctx.close()


def test_in_place_on_another_output(lib):
    bep = lib
    for K in (16, 2000):   # 2000: a reduction in parts
        ctx, cu, se = one_rank(bep, 90, 64, 64)
        x, w, base = ints((90, K), 1), ints((1, K, 48), 2), ints((90, 48), 3, 100)
        y = base.clone()
        bep.bep_ragged_gemm(ctx, cu, se, x, w, y, alpha=2.0, add=y)
        assert bep.bep_status(ctx) == 0
        want = want_y(x, w, np.zeros(90, int), 2.0, base, False)
        assert np.array_equal(bits(y), ref.bf16_bits(want.astype(np.float32)))
        ctx.close()


def test_gradients_against_differences(lib):
    """L = sum c * y is linear in x and in w, and with these integers exact: its differences are the gradients'."""
    bep = lib
    ctx, t = planned(bep, 2, 20, 4, 2, 64, 64, seed=2, skew=0.8)
    rows, K, N = 80, 24, 16
    x, w, c = ints((rows, K), 1, 2), ints((4, K, N), 2, 2), ints((rows, N), 3, 2)
    y, dx, g = torch.empty_like(c), torch.empty_like(x), torch.empty(4, K, N, device=DEV)

    def loss(x, w):
        bep.bep_ragged_gemm(ctx, t["cu"], t["se"], x, w, y)   # |y| <= 24 * 4: exact in bf16
        return (y.double() * c.double()).sum().item()

    base = loss(x, w)
    bep.bep_ragged_gemm(ctx, t["cu"], t["se"], c, w, dx, trans=True)
    bep.bep_ragged_gemm_dw(ctx, t["cu"], t["se"], x, c, g)
    ex, ew = ints((rows, K), 7, 1), ints((4, K, N), 8, 1)
    assert loss(x + ex, w) - base == (dx.double() * ex.double()).sum().item()
    assert loss(x, w + ew) - base == (g.double() * ew.double()).sum().item()
    assert bep.bep_status(ctx) == 0
    ctx.close()


def test_offsets_beyond_32_bits(lib):
    """Rows 32,768 elements apart: the last ones lie more than 2^31 elements behind the first."""
    bep = lib
    rows, K, N, ld = 70000, 72, 40, 32768
    ctx, cu, se = one_rank(bep, rows, 64, 64)
    buf = torch.empty(rows, ld, dtype=torch.bfloat16, device=DEV)
    x, y, add = buf[:, 64:64 + K], buf[:, 1024:1024 + N], buf[:, ld - N:]
    x.copy_(ints((rows, K), 1))
    add.copy_(ints((rows, N), 2, 100))
    w = ints((1, K, N), 3)
    g = torch.empty(1, K, N, device=DEV)
    bep.bep_ragged_gemm(ctx, cu, se, x, w, y, add=add)
    bep.bep_ragged_gemm_dw(ctx, cu, se, x, add, g)
    assert bep.bep_status(ctx) == 0
    want = (x.float() @ w[0].float() + add.float()).bfloat16()
    assert torch.equal(y, want)
    assert torch.equal(g[0].double(), x.double().t() @ add.double())
    ctx.close()


def test_captured_with_a_changing_table(lib):
    """One graph on a side stream, the context's first calls among it; the table changes between replays."""
    bep = lib
    E, K, N, n = 4, 200, 24, 64
    ctx = context(bep, E, E, n)
    cu = torch.zeros(1, 2 * E + 1, dtype=torch.int32, device=DEV)
    se = torch.full((1, E), -1, dtype=torch.int32, device=DEV)
    x, dy, w = ints((n, K), 1), ints((n, N), 2), ints((E, K, N), 3)
    y = torch.empty(n, N, dtype=torch.bfloat16, device=DEV)
    g = torch.empty(E, K, N, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        bep.bep_ragged_gemm(ctx, cu, se, x, w, y)
        bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g)
    for lens in ([10, 20, 30, 4], [0, 0, 64, 0], [1, 0, 0, 0]):
        cu[0, 1:E + 1] = torch.tensor(np.cumsum(lens), dtype=torch.int32)
        cu[0, E + 1:] = sum(lens)
        y.fill_(9.0)
        graph.replay()
        expert = np.concatenate((np.repeat(np.arange(E), lens), np.full(n - sum(lens), -1)))
        want = ref.bf16_bits(want_y(x, w, expert, 1.0, None, False).astype(np.float32))
        assert np.array_equal(bits(y)[expert >= 0], want[expert >= 0])
        assert (y[sum(lens):] == 9).all()
        assert np.array_equal(g.cpu().numpy(), want_g(x, dy, expert, E, 1.0))
    assert bep.bep_status(ctx) == 0
    ctx.close()


def test_adapters_beside_8_bit_experts(lib):
    """A projection in 8 bits with a low-rank adapter on top, as a serving step runs them, and the adapter's
    training step on the same plan."""
    bep = lib
    R, S, E, top, H, Hp, rank = 2, 40, 8, 2, 256, 192, 16
    ctx, t = planned(bep, R, S, E, top, H, Hp, seed=6, skew=1.0)
    expert = row_experts(ctx.cfg, t)
    rows = R * S * top
    gen = torch.Generator(DEV).manual_seed(4)
    x = torch.randn(R, S, H, device=DEV, generator=gen).bfloat16()
    w = (torch.randn(E, H, Hp, device=DEV, generator=gen) * H ** -0.5).bfloat16()
    A = (torch.randn(E, H, rank, device=DEV, generator=gen) * H ** -0.5).bfloat16()
    Bm = torch.randn(E, rank, Hp, device=DEV, generator=gen).bfloat16()
    q, r = bep.IntWeight(ctx), bep.IntRows(rows, H)
    bep.bep_int_quantize_weight(ctx, w, q.codes, q.scales)
    recv = torch.empty(rows, H, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(rows, Hp, dtype=torch.bfloat16, device=DEV)
    h = torch.empty(rows, rank, dtype=torch.bfloat16, device=DEV)
    bep.bep_dispatch(ctx, x, t["dest"], recv)
    bep.bep_dispatch_int(ctx, x, t["dest"], r.codes, r.scales)
    bep.bep_grouped_gemm_int(ctx, t["cu"], t["se"], r.codes, r.scales, q.codes, q.scales, y)
    base = y.clone()
    bep.bep_ragged_gemm(ctx, t["cu"], t["se"], recv, A, h)
    bep.bep_ragged_gemm(ctx, t["cu"], t["se"], h, Bm, y, alpha=0.25, add=y)
    want = want_y(h, Bm, expert, 0.25, base, False)
    mag = want_y(h.abs(), Bm.abs(), expert, 0.25, base.abs(), False)
    assert np.all(np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -22 * mag)
    # against the unquantised layer: 8-bit rows and weights are off by 1/254 of their largest (about 3.5 sigma) at
    # most, uniformly: 0.4% of the output's size each
    full = want_y(recv, w, expert, 1.0, None, False)
    full += want_y(recv, torch.einsum("ehr,ern->ehn", A.float(), Bm.float()), expert, 0.25, None, False)
    err = np.linalg.norm(f64(y) - full) / np.linalg.norm(full)
    assert err < 0.02, err
    # training: gradients of both factors and of the rows
    dy = torch.randn(rows, Hp, device=DEV, generator=gen).bfloat16()
    dh, dx = torch.empty_like(h), torch.empty_like(recv)
    gA, gB = torch.empty(E, H, rank, device=DEV), torch.empty(E, rank, Hp, device=DEV)
    bep.bep_ragged_gemm(ctx, t["cu"], t["se"], dy, Bm, dh, trans=True, alpha=0.25)
    bep.bep_ragged_gemm_dw(ctx, t["cu"], t["se"], h, dy, gB, alpha=0.25)
    bep.bep_ragged_gemm(ctx, t["cu"], t["se"], dh, A, dx, trans=True)
    bep.bep_ragged_gemm_dw(ctx, t["cu"], t["se"], recv, dh, gA)
    assert bep.bep_status(ctx) == 0
    leaves = [v.double().requires_grad_() for v in (recv, A, Bm)]
    e = torch.from_numpy(expert).to(DEV)
    hh = torch.einsum("nh,nhr->nr", leaves[0], leaves[1][e])
    out = 0.25 * torch.einsum("nr,nrk->nk", hh, leaves[2][e])
    want = torch.autograd.grad(out, leaves, dy.double())
    for got, ww in zip((dx, gA, gB), want):
        # each factor passes through one or two bf16 roundings (2^-9 of its size on average)
        assert ((got.double() - ww).norm() / ww.norm()).item() < 2.0 ** -7
    ctx.close()


def test_refusals(lib):
    bep = lib
    ctx, cu, se = one_rank(bep, 8, 64, 64)
    x, w, y = ints((8, 16), 1), ints((1, 16, 24), 2), ints((8, 24), 3)
    g = torch.empty(1, 16, 24, device=DEV)

    def refused(code, f, *a, **k):
        with pytest.raises(bep.BepError) as e:
            f(ctx, cu, se, *a, **k)
        assert e.value.code == code

    arg, al = bep.BEP_ERR_ARG, bep.BEP_ERR_ALIGN
    gemm, dw = bep.bep_ragged_gemm, bep.bep_ragged_gemm_dw
    refused(arg, gemm, ints((8, 12), 1), ints((1, 12, 24), 2), y)                        # widths of 12 and 20
    refused(arg, gemm, x, ints((1, 16, 20), 2), ints((8, 20), 3))
    refused(arg, gemm, ints((8, 28), 1)[:, :16], w, y)                                   # rows 28 apart
    refused(arg, gemm, ints((1, 16), 1).expand(8, 16), w, y)                             # rows on one another
    refused(al, gemm, ints((8, 32), 1)[:, 4:20], w, y)
    refused(arg, gemm, x, w, y, alpha=float("nan"))
    refused(arg, gemm, x, w, y, alpha=float("inf"))
    refused(arg, gemm, x, ints((1, 16, 16), 2), x)                                       # onto its own input
    both = ints((8, 48), 4)
    refused(arg, gemm, x, w, both[:, :24], add=both.view(-1)[:192].view(8, 24))          # in place, other strides
    refused(arg, dw, ints((8, 12), 1), y, torch.empty(1, 12, 24, device=DEV))
    for bad, kind in ((dict(x=x.float()), TypeError), (dict(x=x[:7]), ValueError), (dict(w=w[0]), ValueError),
                      (dict(w=w.transpose(1, 2)), ValueError), (dict(y=y.t().contiguous().t()), ValueError),
                      (dict(add=ints((8, 32), 1)), ValueError), (dict(x=x.cpu()), ValueError), (dict(w=w.half()), TypeError)):
        with pytest.raises(kind):
            gemm(ctx, cu, se, **{**dict(x=x, w=w, y=y), **bad})
    with pytest.raises(ValueError):
        dw(ctx, cu, se, x, y, g[:, :8])
    with pytest.raises(TypeError):
        dw(ctx, cu, se, x, y, g.bfloat16())
    ctx.close()


def test_calls_without_tokens(lib):
    bep = lib
    ctx = bep.Context(bep.Config(2, 4, 2, 1, 0, 64, 64, bep.BEP_TRAIN))
    L = bep.load()
    assert L.bep_ragged_gemm(ctx.handle, None, None, None, 8, 8, None, 8, 0, 1.0, None, 0, None, 8, None) == 0
    g = torch.full((4, 8, 16), 9.0, device=DEV)
    assert L.bep_ragged_gemm_dw(ctx.handle, None, None, None, 8, 8, None, 16, 16, 1.0, 1, g.data_ptr(), None) == 0
    assert (g == 9).all()
    assert L.bep_ragged_gemm_dw(ctx.handle, None, None, None, 8, 8, None, 16, 16, 1.0, 0, g.data_ptr(), None) == 0
    torch.cuda.synchronize()
    assert (g == 0).all()
    ctx.close()
