"""Grouped products of any width at sizes where pairs of SMs share a unit, and gradients where a unit has two tiles: small
integers, whose sums are exact in fp32 in any order, to the bit."""
import pytest
import torch

from kernel_forms import expect
from test_gpu_int8 import bits
from test_gpu_ragged import context, ints, table, wide

pytestmark = pytest.mark.gpu
DEV = "cuda"

# tiles of 256 rows: last ones of 1, 16, 17, 64, 127, 128, 129, 255 and 256 rows, an expert without rows
PAIR_LENS = [4097, 4112, 0, 4113, 4160, 4223, 4224, 4225, 4351, 4352]


def spans(lens):
    at = 0
    for e, n in enumerate(lens):
        yield e, slice(at, at + n)
        at += n


def exact_rows(x, w, lens, alpha, trans, out):
    for e, at in spans(lens):
        if at.stop > at.start:
            m = w[e].double()
            out[at] = (alpha * (x[at].double() @ (m.t() if trans else m))).float().bfloat16()
    return out


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K,N,pad", [
    (576, 136, 64),     # nine blocks in two chains, one tile of columns, rows that start on whole lines
    (520, 264, 24),     # a last block of 8, two tiles
    (1032, 520, 24),    # three chains, three tiles
    (1096, 1096, 8),    # more blocks than the ring has stages, five tiles
    (1600, 256, 0),     # one full tile
    (1024, 2048, 64),   # eight full tiles
])
def test_products_on_pairs_of_SMs(lib, K, N, pad, trans):
    """With NaN in single rows, whose outputs alone are NaN, a slot without an expert and rows behind the last segment."""
    bep = lib
    E = len(PAIR_LENS)
    cu, se, n = table(PAIR_LENS, slots=[(99, 300)], spare=45)
    ctx = context(bep, E, 1, n)
    x, _ = wide(ints((n, K), 1), pad, 0)
    w = ints((E, N, K) if trans else (E, K, N), 2)
    used = sum(PAIR_LENS)
    nan = [0, 4096, 4097, 8208, used - 1]      # the first and the last rows of segments
    x[nan] = float("nan")
    x[used:] = float("nan")
    y, yb = wide(torch.full((n, N), 9.0, dtype=torch.bfloat16, device=DEV), 24, 16, 9.0)
    want = torch.full((n, N), 9.0, dtype=torch.bfloat16, device=DEV)
    exact_rows(torch.nan_to_num(x), w, PAIR_LENS, 0.25, trans, want)
    want[nan] = float("nan")
    form = "ragged_kernel<%s, false, 16, true>" % ("true" if trans else "false")
    expect(lambda: bep.bep_ragged_gemm(ctx, cu, se, x, w, y, trans=trans, alpha=0.25), form)
    for _ in range(2):
        assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
        bep.bep_clear_status(ctx)
        assert y[nan].isnan().all()
        ok = torch.ones(n, dtype=torch.bool, device=DEV)
        ok[nan] = False
        assert torch.equal(y[ok], want[ok])
        assert (yb[:, :24] == 9).all() and (yb[:, 24 + N:] == 9).all()
        y[:used].fill_(9.0)
        bep.bep_ragged_gemm(ctx, cu, se, x, w, y, trans=trans, alpha=0.25)
    ctx.close()


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("K,N,add,form", [
    (528, 1544, False, "16, false"), (2056, 1544, True, "16, false"), (528, 104, True, "8, false"), (2056, 72, False, "8, false"),
    (512, 1544, False, "0, false"), (512, 104, True, "0, false"),
])
def test_products_around_a_chain(lib, K, N, add, form, trans):
    """The same segments, shorter, on single SMs."""
    bep = lib
    lens = [max(n - 3900, 0) for n in PAIR_LENS]
    E = len(lens)
    cu, se, n = table(lens, slots=[(99, 30)], spare=45)
    ctx = context(bep, E, 1, n)
    x, _ = wide(ints((n, K), 1), 8, 0)
    w = ints((E, N, K) if trans else (E, K, N), 2)
    base = ints((n, N), 3, 100) if add else None
    y = torch.full((n, N), 9.0, dtype=torch.bfloat16, device=DEV)
    want = y.clone()
    for e, at in spans(lens):
        if at.stop > at.start:
            v = x[at].double() @ (w[e].double().t() if trans else w[e].double())
            want[at] = (-0.5 * v + (base[at].double() if add else 0)).float().bfloat16()
    name = "ragged_kernel<%s, %s, %s>" % ("true" if trans else "false", "true" if add else "false", form)
    expect(lambda: bep.bep_ragged_gemm(ctx, cu, se, x, w, y, trans=trans, alpha=-0.5, add=base), name)
    assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
    assert torch.equal(y, want)
    ctx.close()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("K,N", [(1288, 16), (1288, 72), (1288, 128), (16, 1288), (72, 1288), (2048, 24)])
def test_gradients_of_two_tiles_a_unit(lib, K, N, accumulate):
    """One of the widths narrow and many experts; the last unit of 1288 has a part of its first tile alone. Rows behind
    each segment are another's, those behind the last NaN."""
    bep = lib
    gen = torch.Generator().manual_seed(K + N)
    lens = torch.randint(0, 90, (64,), generator=gen).tolist()
    lens[5] = lens[63] = 0
    lens[20] = 700
    E = len(lens)
    cu, se, n = table(lens, slots=[(3, 75)], spare=40)
    ctx = context(bep, E, 1, n)
    x, dy = wide(ints((n, K), 1), 8, 16)[0], wide(ints((n, N), 2), 24, 0)[0]
    used = sum(lens) + 75
    x[used:], dy[used:] = float("nan"), float("nan")
    want = torch.full((E, K, N), 3.0 if accumulate else 0.0, dtype=torch.float64, device=DEV)
    for e, at in [*spans(lens), (3, slice(used - 75, used))]:
        want[e] += 0.5 * (x[at].double().t() @ dy[at].double())
    raw = torch.full((E * K * N + 2048,), 3.0, device=DEV)
    g = raw[1024:1024 + E * K * N].view(E, K, N)
    expect(lambda: bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g, alpha=0.5, accumulate=accumulate), "ragged_dw_kernel<2, false>")
    assert bep.bep_status(ctx) == 0
    assert torch.equal(g.double(), want)
    assert (raw[:1024] == 3).all() and (raw[-1024:] == 3).all()
    ctx.close()


def test_two_streams_of_pairs(lib):
    """Two contexts on two streams, both products on pairs of SMs, against the same calls one after another."""
    bep = lib
    cu, se, n = table(PAIR_LENS, slots=[(1, 300)])
    E, K, N = len(PAIR_LENS), 776, 776
    both = []
    for i in range(2):
        ctx = context(bep, E, 1, n)
        x, w = ints((n, K), 10 + i), ints((E, K, N), 20 + i)
        y = [torch.empty(n, N, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        bep.bep_ragged_gemm(ctx, cu, se, x, w, y[0])
        both.append((ctx, x, w, y))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(3):
        for s, (ctx, x, w, y) in zip(streams, both):
            bep.bep_ragged_gemm(ctx, cu, se, x, w, y[1], stream=s)
    torch.cuda.synchronize()
    for ctx, x, w, y in both:
        assert bep.bep_status(ctx) == 0
        assert (bits(y[0]) == bits(y[1])).all()
        ctx.close()


def test_captured_pairs_with_a_changing_table(lib):
    """A graph of a product on pairs of SMs and its matrices' gradient, whose table changes between replays: other lengths,
    no rows at all, a table that is refused."""
    bep = lib
    cu, se, n = table(PAIR_LENS, slots=[(1, 300)])
    E, K, N = len(PAIR_LENS), 584, 264
    ctx = context(bep, E, 1, n)
    x, w, dy = ints((n, K), 1), ints((E, K, N), 2), ints((n, N), 3)
    y = torch.empty(n, N, dtype=torch.bfloat16, device=DEV)
    g = torch.empty(E, K, N, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        bep.bep_ragged_gemm(ctx, cu, se, x, w, y)
        bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g)
    for lens in (PAIR_LENS, PAIR_LENS[::-1], [0] * E, [n] + [0] * (E - 1), [1] * E):
        at = torch.tensor([0, *lens, 0]).cumsum(0)
        cu[0] = at.to(torch.int32)
        y.fill_(9.0)
        graph.replay()
        assert bep.bep_status(ctx) == 0
        want = exact_rows(x, w, lens, 1.0, False, torch.full_like(y, 9.0))
        assert torch.equal(y, want)
        for e, rows in spans(lens):
            assert torch.equal(g[e].double(), x[rows].double().t() @ dy[rows].double())
    cu[0, 3] = n + 1
    y.fill_(9.0)
    g.fill_(9.0)
    graph.replay()
    assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
    assert (y == 9).all() and (g == 9).all()
    ctx.close()
