"""The 8-bit and the any-width products among other work: tables and rows that the kernel in front is still writing,
two contexts on two streams, many calls in a row without a synchronisation."""
import numpy as np
import pytest
import torch

import int8_ref as ref
from test_gpu_int8 import bits, weights
from test_gpu_ragged import ints, want_g, want_y

pytestmark = pytest.mark.gpu
DEV = "cuda"
E, H, HP, K, N = 6, 256, 128, 200, 72


def tables(rows, count, seed):
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(count):
        cu = np.zeros((1, 2 * E + 1), np.int32)
        cu[0, 1:E + 1] = np.sort(rng.integers(0, rows + 1, size=E))
        cu[0, E + 1:] = cu[0, E]
        out.append(cu)
    return out


def experts(cu, rows):
    e = np.full(rows, -1)
    for i in range(E):
        e[cu[0, i]:cu[0, i + 1]] = i
    return e


# rows: the call makes its own list of row tiles, or has a kernel make it
@pytest.mark.parametrize("rows", [60, 3000, 40000])
def test_tables_and_rows_written_just_before(lib, rows):
    bep = lib
    ctx = bep.Context(bep.Config(1, E, E, 1, rows, H, HP, bep.BEP_TRAIN))
    w8, w = weights(bep, ctx), ints((E, K, N), 1)
    se = torch.full((1, E), -1, dtype=torch.int32, device=DEV)
    cu = torch.zeros(1, 2 * E + 1, dtype=torch.int32, device=DEV)
    dest = torch.arange(rows, dtype=torch.int32, device=DEV).view(1, rows, 1)
    x8, x, dy = torch.empty(1, rows, H, device=DEV).bfloat16(), ints((rows, K), 2), ints((rows, N), 3)
    src8 = [torch.randn(1, rows, H, device=DEV, generator=torch.Generator(DEV).manual_seed(i)).bfloat16() for i in range(4)]
    src = [ints((rows, K), 10 + i) for i in range(4)]
    tab = tables(rows, 4, rows)
    dtab = [torch.from_numpy(t).to(DEV) for t in tab]
    q, y8 = bep.IntRows(rows, H), torch.zeros(rows, HP, dtype=torch.bfloat16, device=DEV)
    y, g = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV), torch.empty(E, K, N, device=DEV)
    got = []
    for i in range(12):
        k = i % 4
        cu.copy_(dtab[k])
        x8.copy_(src8[k])
        bep.bep_dispatch_int(ctx, x8, dest, q.codes, q.scales)
        bep.bep_grouped_gemm_int(ctx, cu, se, q.codes, q.scales, w8.codes, w8.scales, y8)
        x.copy_(src[k])
        bep.bep_ragged_gemm(ctx, cu, se, x, w, y)
        bep.bep_ragged_gemm_dw(ctx, cu, se, x, dy, g)
        got.append((y8.clone(), y.clone(), g.clone()))
    assert bep.bep_status(ctx) == 0
    wq, ws = w8.codes.cpu().numpy(), w8.scales.cpu().numpy()
    for i, (a, b, c) in enumerate(got):
        k = i % 4
        e = experts(tab[k], rows)
        assert np.array_equal(c.cpu().numpy(), want_g(src[k], dy, e, E, 1.0)), i
        at = e >= 0
        assert np.array_equal(bits(b)[at], ref.bf16_bits(want_y(src[k], w, e, 1.0, None, False).astype(np.float32))[at]), i
        codes, scales = ref.quantise(src8[k].double().cpu().numpy()[0])
        for j in range(E):
            r = e == j
            if r.any():
                assert np.array_equal(bits(a)[r], ref.product_bits(codes[r], scales[r], wq[j], ws[j])), (i, j)
    ctx.close()


def test_two_contexts_on_two_streams(lib):
    bep = lib
    rows = 900
    sides = []
    for seed in (1, 2):
        ctx = bep.Context(bep.Config(1, E, E, 1, rows, H, HP, bep.BEP_TRAIN))
        cu = tables(rows, 1, seed)[0]
        s = dict(ctx=ctx, cu=torch.from_numpy(cu).to(DEV), se=torch.full((1, E), -1, dtype=torch.int32, device=DEV),
                 x=ints((rows, K), seed), w=ints((E, K, N), seed + 5), dy=ints((rows, N), seed + 9), stream=torch.cuda.Stream(),
                 y=torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV), g=torch.empty(E, K, N, device=DEV),
                 w8=weights(bep, ctx, seed), q=bep.IntRows(rows, H), y8=torch.zeros(rows, HP, dtype=torch.bfloat16, device=DEV))
        s["q"].codes.copy_(torch.randint(-127, 128, (rows, H), device=DEV))
        s["q"].scales.fill_(0.5)
        sides.append(s)

    def step(s, stream):
        bep.bep_ragged_gemm(s["ctx"], s["cu"], s["se"], s["x"], s["w"], s["y"], stream=stream)
        bep.bep_grouped_gemm_int(s["ctx"], s["cu"], s["se"], s["q"].codes, s["q"].scales, s["w8"].codes, s["w8"].scales, s["y8"],
                                 stream=stream)
        bep.bep_ragged_gemm_dw(s["ctx"], s["cu"], s["se"], s["x"], s["dy"], s["g"], stream=stream)

    torch.cuda.synchronize()
    want = []
    for s in sides:
        step(s, None)
        torch.cuda.synchronize()
        want.append([s[n].clone() for n in ("y", "y8", "g")])
        for n in ("y", "y8", "g"):
            s[n].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s in sides:
            step(s, s["stream"])
    torch.cuda.synchronize()
    for s, v in zip(sides, want):
        assert bep.bep_status(s["ctx"]) == 0
        for n, t in zip(("y", "y8", "g"), v):
            assert torch.equal(s[n].float(), t.float()), n
        s["ctx"].close()


def test_outputs_beyond_32_bit_offsets(lib):
    """2.3e9 outputs and weights: rows and channels at the far end, against the first ones' exact sums."""
    bep = lib
    rows, H_, Hp = 320000, 64, 7168
    ctx = bep.Context(bep.Config(1, 1, 1, 1, rows, H_, Hp, bep.BEP_TRAIN))
    cu = torch.tensor([[0, rows, rows]], dtype=torch.int32, device=DEV)
    se = torch.full((1, 1), -1, dtype=torch.int32, device=DEV)
    w, q = weights(bep, ctx), bep.IntRows(rows, H_)
    q.codes.copy_(torch.randint(-127, 128, (rows, H_), device=DEV, dtype=torch.int8))
    q.scales.copy_(torch.rand(rows, device=DEV) + 0.5)
    y = torch.empty(rows, Hp, dtype=torch.bfloat16, device=DEV)
    bep.bep_grouped_gemm_int(ctx, cu, se, q.codes, q.scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0
    at = torch.tensor([0, 1, 127, 255, 256, 299999, 300032, 319998, 319999], device=DEV)
    want = ref.product_bits(q.codes[at].cpu().numpy(), q.scales[at].cpu().numpy(), w.codes[0].cpu().numpy(), w.scales[0].cpu().numpy())
    assert np.array_equal(bits(y[at]), want)
    ctx.close()
    del w, q, y
    E_, H_, Hp = 330, 1024, 7168        # the last expert's codes begin beyond 2^31 bytes
    ctx = bep.Context(bep.Config(1, E_, E_, 1, 40, H_, Hp, bep.BEP_TRAIN))
    cu = torch.zeros(1, 2 * E_ + 1, dtype=torch.int32, device=DEV)
    cu[0, E_:] = 40
    se = torch.full((1, E_), -1, dtype=torch.int32, device=DEV)
    w, q = bep.IntWeight(ctx), bep.IntRows(40, H_)
    full = torch.randn(E_, H_, Hp, device=DEV, dtype=torch.bfloat16) * 0.02
    bep.bep_int_quantize_weight(ctx, full, w.codes, w.scales)
    last = full[-1].double().cpu().numpy().T
    codes, scales = ref.quantise(last)
    assert np.array_equal(w.codes[-1].cpu().numpy(), codes) and np.array_equal(w.scales[-1].cpu().numpy(), scales)
    q.codes.copy_(torch.randint(-127, 128, (40, H_), device=DEV, dtype=torch.int8))
    q.scales.fill_(1.0)
    y = torch.empty(40, Hp, dtype=torch.bfloat16, device=DEV)
    bep.bep_grouped_gemm_int(ctx, cu, se, q.codes, q.scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0
    assert np.array_equal(bits(y), ref.product_bits(q.codes.cpu().numpy(), np.ones(40, np.float32), codes, scales))
    ctx.close()
