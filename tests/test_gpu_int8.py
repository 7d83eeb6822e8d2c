"""Experts in 8-bit integers on the GPU against a 64-bit reference: codes and scales exactly, products to the
bit where their sums stay below 2^24, else within fp32 accumulation and one bf16 rounding."""
import numpy as np
import pytest
import torch

import experts_ref
import int8_ref as ref
from test_gpu_mx import bf16, f64, planned, row_experts

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def weights(bep, ctx, seed=1):
    c = ctx.cfg
    rng = np.random.default_rng([seed, c.H, c.Hp])
    w = bf16(rng.normal(size=(c.E, c.H, c.Hp)) * 0.02)
    q = bep.IntWeight(ctx)
    bep.bep_int_quantize_weight(ctx, w, q.codes, q.scales)
    return q


def one_rank(bep, rows, H, Hp, E=1):
    """A context whose receive rows are `rows` rows, and a table that gives them all to expert 0."""
    ctx = bep.Context(bep.Config(1, E, E, 1, rows, H, Hp, bep.BEP_TRAIN))
    cu = torch.zeros(1, 2 * E + 1, dtype=torch.int32, device=DEV)
    cu[0, 1:] = rows
    return ctx, cu, torch.full((1, E), -1, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("E,H,Hp", [(2, 64, 64), (3, 128, 192), (2, 1088, 576), (1, 4160, 128)])
def test_weight_quantisation(lib, E, H, Hp):
    bep = lib
    ctx = bep.Context(bep.Config(1, E, E, 1, 4, H, Hp, bep.BEP_TRAIN))
    rng = np.random.default_rng([E, H])
    v = rng.normal(size=(E, H, Hp)) * np.exp2(rng.integers(-20, 20, size=(E, 1, Hp)))
    v[0, :, 0] = 0
    v[0, 5, 1], v[0, 7, 1] = np.inf, -np.inf
    v[0, 6, 2] = np.nan
    v[0, :, 3] = 1e-39 * rng.normal(size=H)           # subnormal numbers
    v[0, :, 4] = 3.3e38 * np.sign(v[0, :, 5])
    v[0, :, 6] = np.arange(H) % 128 - 63.5            # with 127: 127 v / m ties (m = 127, v = k + 1/2)
    v[0, 3, 6] = -127
    v[0, :, 7] = 0.5
    v[0, 0, 7] = 1.0                                  # 63.5
    v[0, :, 8] = 1e-30 * v[0, :, 9]
    v[0, 0, 8] = 1e30                                 # the others are 0 beside it
    w = bf16(v)
    raw = torch.full((E * Hp * H + 4096,), 0x55, dtype=torch.int8, device=DEV)
    codes = raw[2048:2048 + E * Hp * H].view(E, Hp, H)
    q = bep.IntWeight(ctx)
    bep.bep_int_quantize_weight(ctx, w, codes, q.scales)
    assert bep.bep_status(ctx) == 0
    assert (raw[:2048] == 0x55).all() and (raw[-2048:] == 0x55).all()
    wc, ws = ref.quantise(f64(w).transpose(0, 2, 1))
    assert np.array_equal(q.scales.cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(codes.cpu().numpy(), wc)
    ctx.close()


# widths: one piece of 16, a CTA's two held rounds, and a part that is read again (beyond 16384)
@pytest.mark.parametrize("R,S,E,K,H", [(1, 1, 8, 3, 64), (2, 33, 8, 2, 1088), (1, 2, 40, 32, 7168), (1, 3, 4, 2, 8256),
                                       (1, 2, 4, 3, 20544)])
def test_dispatch_in_8_bits(lib, R, S, E, K, H):
    bep = lib
    ctx, t = planned(bep, R, S, E, K, H, 64)
    rng = np.random.default_rng([S, H])
    v = rng.normal(size=(R * S, H)) * np.exp2(rng.integers(-8, 8, size=(R * S, 1)))
    v[-1, 1:] = v[-1, 0] / 2                          # ties at 63.5
    if S > 2:
        v[0, H - 1] = np.inf
        v[1] = 0
    x = bf16(v).view(R, S, H)
    n = R * S * K
    raw = torch.full((n * H + 4096,), 0x55, dtype=torch.int8, device=DEV)
    codes = raw[2048:2048 + n * H].view(n, H)
    scales = torch.full((n,), -1.0, device=DEV)
    bep.bep_dispatch_int(ctx, x, t["dest"], codes, scales)
    assert bep.bep_status(ctx) == 0
    assert (raw[:2048] == 0x55).all() and (raw[-2048:] == 0x55).all()
    wc, ws = ref.quantise(f64(x).reshape(R * S, H))
    dest = t["dest"].cpu().numpy().reshape(R * S, K)
    for k in range(K):
        assert np.array_equal(codes.cpu().numpy()[dest[:, k]], wc)
        assert np.array_equal(scales.cpu().numpy()[dest[:, k]], ws, equal_nan=True)
    ctx.close()


@pytest.mark.parametrize("H", [128, 20544])
def test_dispatch_skips_bad_destinations(lib, H):
    bep = lib
    ctx, t = planned(bep, 2, 16, 8, 2, H, 64)
    dest = t["dest"].clone()
    dest[0, 3, 1], dest[1, 0, 0] = 64, -1
    raw = torch.full((64 * H + 8192,), 0x33, dtype=torch.int8, device=DEV)
    rows = bep.IntRows(64, H)
    bep.bep_dispatch_int(ctx, torch.ones(2, 16, H, dtype=torch.bfloat16, device=DEV), dest,
                         raw[4096:4096 + 64 * H].view(64, H), rows.scales)
    assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
    assert (raw[:4096] == 0x33).all() and (raw[-4096:] == 0x33).all()
    ctx.close()


def test_dispatch_under_an_sm_budget(lib):
    bep = lib
    ctx, t = planned(bep, 2, 700, 8, 2, 320, 64)
    x = torch.randn(2, 700, 320, device=DEV).bfloat16()
    a, b = bep.IntRows(2800, 320), bep.IntRows(2800, 320)
    bep.bep_dispatch_int(ctx, x, t["dest"], a.codes, a.scales)
    bep.bep_set_comm_sms(ctx, 3)
    bep.bep_dispatch_int(ctx, x, t["dest"], b.codes, b.scales)
    assert bep.bep_status(ctx) == 0
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    ctx.close()


# widths: one warp a row up to a CTA's eight, and beyond 8192 a part that is made again
@pytest.mark.parametrize("rows,F", [(1, 64), (37, 1088), (3000, 512), (3000, 1024), (2500, 1600), (5, 8192), (3, 8256),
                                    (2, 17408)])
def test_activation_in_8_bits(lib, rows, F):
    bep = lib
    ctx = bep.Context(bep.Config(1, 1, 1, 1, rows, 64, 64, bep.BEP_TRAIN))
    rng = np.random.default_rng([rows, F])
    v = rng.normal(size=(rows, 2 * F)) * 2
    if rows > 2:
        v[1] = 0
        v[2, F - 1] = np.nan
    h = bf16(v)
    raw = torch.full((rows * F + 4096,), 0x55, dtype=torch.int8, device=DEV)
    codes, scales = raw[2048:2048 + rows * F].view(rows, F), torch.full((rows,), -1.0, device=DEV)
    bep.bep_swiglu_int(ctx, h, codes, scales)
    assert bep.bep_status(ctx) == 0
    assert (raw[:2048] == 0x55).all() and (raw[-2048:] == 0x55).all()
    a = experts_ref.swiglu(f64(h))
    wc, ws = ref.quantise(a)
    sc = scales.cpu().numpy()
    # fp32 sigmoid and products, a few units in the last place: 2^-20
    assert np.array_equal(np.isnan(sc), np.isnan(ws))
    assert np.all(np.isnan(ws) | (np.abs(sc - ws) <= 2.0 ** -20 * ws))
    bad = ~np.isfinite(a).all(1)
    m = np.abs(np.where(bad[:, None], 0, a)).max(1, keepdims=True)
    t = 127 * np.where(bad[:, None], 0, a) / np.where(m > 0, m, 1)
    near = np.abs(np.abs(t) % 1 - 0.5) < 127 * 2.0 ** -19      # may go to either side
    got = codes.cpu().numpy().astype(np.int64)
    assert np.all((got == wc) | (near & (np.abs(got - wc) <= 1)))
    ctx.close()


# R, S, E, K, H, H', B (None: training), routing skew
PRODUCTS = [
    (1, 1, 4, 1, 64, 64, None, 0.0),
    (1, 1, 8, 3, 256, 128, None, 0.0),
    (2, 1, 16, 4, 320, 192, None, 0.0),
    (2, 64, 8, 2, 128, 64, None, 1.2),
    (1, 300, 2, 1, 512, 128, None, 0.0),
    (3, 70, 12, 5, 1088, 576, None, 1.0),
    (4, 100, 16, 3, 768, 320, 2, 1.5),
    (8, 17, 24, 6, 4160, 256, 1, 1.5),
    (2, 500, 6, 2, 576, 704, None, 0.3),
    (1, 129, 1, 1, 64, 2048, None, 0.0),
    (1, 257, 1, 1, 192, 256, None, 0.0),
    (1, 1100, 1, 1, 128, 5120, None, 0.0),
    (4, 900, 8, 2, 448, 1088, None, 0.5),
]


@pytest.mark.parametrize("R,S,E,K,H,Hp,B,skew", PRODUCTS)
def test_product(lib, R, S, E, K, H, Hp, B, skew):
    bep = lib
    ctx, t = planned(bep, R, S, E, K, H, Hp, B, seed=3, skew=skew)
    w = weights(bep, ctx)
    rng = np.random.default_rng([R, S, H])
    x = bf16(rng.normal(size=(R, S, H)))
    rows = bep.IntRows(R * S * K, H)
    bep.bep_dispatch_int(ctx, x, t["dest"], rows.codes, rows.scales)
    raw = torch.full((R * S * K * Hp + 8192,), 9.0, dtype=torch.bfloat16, device=DEV)
    y = raw[4096:4096 + R * S * K * Hp].view(R * S * K, Hp)
    bep.bep_grouped_gemm_int(ctx, t["cu"], t["se"], rows.codes, rows.scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0
    assert (raw[:4096] == 9).all() and (raw[-4096:] == 9).all()
    q, s = rows.codes.cpu().numpy(), rows.scales.cpu().numpy()
    wq, ws = w.codes.cpu().numpy(), w.scales.cpu().numpy()
    expert = row_experts(ctx.cfg, t)
    assert (expert >= 0).all()
    got = bits(y)
    for e in np.unique(expert):
        at = expert == e
        assert np.array_equal(got[at], ref.product_bits(q[at], s[at], wq[e], ws[e])), f"expert {e}"
    # the same call again gives the same bits
    y2 = torch.empty_like(y)
    bep.bep_grouped_gemm_int(ctx, t["cu"], t["se"], rows.codes, rows.scales, w.codes, w.scales, y2)
    assert torch.equal(y2.view(torch.int16), y.view(torch.int16))
    ctx.close()


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 64, 65, 96, 127, 128, 129, 160, 224, 255, 256, 257, 288, 385, 512])
def test_product_of_every_tile_height(lib, rows):
    bep = lib
    ctx, cu, se = one_rank(bep, rows, 192, 320)
    w = weights(bep, ctx)
    rng = np.random.default_rng(rows)
    codes = torch.from_numpy(rng.integers(-127, 128, size=(rows, 192)).astype(np.int8)).to(DEV)
    scales = torch.from_numpy(rng.uniform(0.5, 2, size=rows).astype(np.float32)).to(DEV)
    y = torch.empty(rows, 320, dtype=torch.bfloat16, device=DEV)
    bep.bep_grouped_gemm_int(ctx, cu, se, codes, scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0
    want = ref.product_bits(codes.cpu().numpy(), scales.cpu().numpy(), w.codes.cpu().numpy()[0], w.scales.cpu().numpy()[0])
    assert np.array_equal(bits(y), want)
    ctx.close()


def test_units_of_both_accumulator_kinds_in_one_launch(lib):
    """Segments of 1 to 600 rows side by side: units of one accumulator and of both alternate on every pair."""
    bep = lib
    E, H, Hp = 96, 128, 64
    rng = np.random.default_rng(5)
    lens = rng.choice([0, 1, 40, 100, 128, 129, 200, 256, 300, 600], size=E)
    rows = int(lens.sum())
    ctx = bep.Context(bep.Config(1, E, E, 1, rows, H, Hp, bep.BEP_TRAIN))
    cu = torch.zeros(1, 2 * E + 1, dtype=torch.int32, device=DEV)
    cu[0, 1:E + 1] = torch.from_numpy(np.cumsum(lens)).to(DEV)
    cu[0, E + 1:] = rows
    se = torch.full((1, E), -1, dtype=torch.int32, device=DEV)
    w = weights(bep, ctx)
    codes = torch.from_numpy(rng.integers(-127, 128, size=(rows, H)).astype(np.int8)).to(DEV)
    scales = torch.from_numpy(rng.uniform(0.5, 2, size=rows).astype(np.float32)).to(DEV)
    y = torch.empty(rows, Hp, dtype=torch.bfloat16, device=DEV)
    bep.bep_grouped_gemm_int(ctx, cu, se, codes, scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0
    got, q, s = bits(y), codes.cpu().numpy(), scales.cpu().numpy()
    wq, ws = w.codes.cpu().numpy(), w.scales.cpu().numpy()
    at = 0
    for e, n in enumerate(lens):
        assert np.array_equal(got[at:at + n], ref.product_bits(q[at:at + n], s[at:at + n], wq[e], ws[e])), e
        at += n
    ctx.close()


# few units for the pairs of SMs: the reduction is cut into parts, for all units or for those of the last round
@pytest.mark.parametrize("R,S,E,K,H,Hp", [(1, 1, 8, 3, 7168, 64), (1, 1, 4, 1, 576, 320), (1, 2, 40, 4, 7168, 2048), (8, 1, 64, 4, 3712, 1024),
                                          (1, 33, 1, 1, 5120, 512), (2, 30, 2, 1, 2048, 10496)])
def test_few_units(lib, R, S, E, K, H, Hp):
    bep = lib
    ctx, t = planned(bep, R, S, E, K, H, Hp, seed=4, skew=0.3)
    w = weights(bep, ctx)
    rng = np.random.default_rng([S, H])
    x = bf16(rng.normal(size=(R, S, H)))
    rows = bep.IntRows(R * S * K, H)
    bep.bep_dispatch_int(ctx, x, t["dest"], rows.codes, rows.scales)
    q, s = rows.codes.cpu().numpy(), rows.scales.cpu().numpy()
    wq, ws = w.codes.cpu().numpy(), w.scales.cpu().numpy()
    expert = row_experts(ctx.cfg, t)
    want = np.zeros((R * S * K, Hp), np.uint16)
    for e in np.unique(expert):
        want[expert == e] = ref.product_bits(q[expert == e], s[expert == e], wq[e], ws[e])
    for _ in range(3):
        y = torch.full((R * S * K, Hp), 9.0, dtype=torch.bfloat16, device=DEV)
        bep.bep_grouped_gemm_int(ctx, t["cu"], t["se"], rows.codes, rows.scales, w.codes, w.scales, y)
        assert np.array_equal(bits(y), want)
    assert bep.bep_status(ctx) == 0
    ctx.close()


def test_sums_beyond_24_bits(lib):
    """Every code at its limit, 7168 of them: 127 * 127 * 7168 = 1.2e8. A sum over 16 products at a time that is
    truncated to fp32 after each is off by 2^-23 of the magnitudes for each of the H / 16 steps at most."""
    bep = lib
    rows, H, Hp = 40, 7168, 128
    ctx, cu, se = one_rank(bep, rows, H, Hp)
    rng = np.random.default_rng(8)
    q = np.where(rng.random((rows, H)) < 0.75, 127, -127).astype(np.int8)
    q[:8] = 127
    wq = np.where(rng.random((1, Hp, H)) < 0.75, 127, -127).astype(np.int8)
    wq[0, :8] = 127
    y = torch.empty(rows, Hp, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(rows, device=DEV), torch.ones(1, Hp, device=DEV)
    bep.bep_grouped_gemm_int(ctx, cu, se, torch.from_numpy(q).to(DEV), one[0], torch.from_numpy(wq).to(DEV), one[1], y)
    assert bep.bep_status(ctx) == 0
    want = q.astype(np.float64) @ wq[0].astype(np.float64).T
    mag = 127.0 * 127.0 * H
    assert np.all(np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + (H / 16) * 2.0 ** -23 * mag)
    ctx.close()


def test_nan_rows_and_channels_stay_their_own(lib):
    bep = lib
    rows, H, Hp = 70, 128, 192
    ctx, cu, se = one_rank(bep, rows, H, Hp)
    w = torch.randn(1, H, Hp, device=DEV).bfloat16()
    w[0, 3, 100] = float("inf")
    q = bep.IntWeight(ctx)
    bep.bep_int_quantize_weight(ctx, w, q.codes, q.scales)
    x = torch.randn(1, rows, H, device=DEV).bfloat16()
    x[0, 33, 5] = float("nan")
    x[0, 34] = 0
    r = bep.IntRows(rows, H)
    dest = torch.arange(rows, dtype=torch.int32, device=DEV).view(1, rows, 1)
    bep.bep_dispatch_int(ctx, x, dest, r.codes, r.scales)
    y = torch.empty(rows, Hp, dtype=torch.bfloat16, device=DEV)
    bep.bep_grouped_gemm_int(ctx, cu, se, r.codes, r.scales, q.codes, q.scales, y)
    assert bep.bep_status(ctx) == 0
    nan = torch.zeros(rows, Hp, dtype=torch.bool, device=DEV)
    nan[33], nan[:, 100] = True, True
    assert torch.equal(y.isnan(), nan)
    assert (y[34][~nan[34]] == 0).all()
    ctx.close()


def test_tables_and_rows_that_no_segment_covers(lib):
    """Rows behind the last segment and of a slot without an expert keep what they held; a bad table is refused."""
    bep = lib
    R, S, E, K, H, Hp = 2, 40, 4, 1, 128, 64
    ctx = bep.Context(bep.Config(R, E, 2, K, S, H, Hp, bep.BEP_TRAIN))
    w = weights(bep, ctx)
    rng = np.random.default_rng(4)
    codes = torch.from_numpy(rng.integers(-127, 128, size=(80, H)).astype(np.int8)).to(DEV)
    scales = torch.ones(80, device=DEV)
    cu = torch.tensor([[0, 3, 3, 9, 9, 20, 30], [0, 0, 0, 0, 0, 0, 0]], dtype=torch.int32, device=DEV)
    se = torch.tensor([[2, 7], [-1, -1]], dtype=torch.int32, device=DEV)   # 7: no such expert
    y = torch.full((80, Hp), 5.0, dtype=torch.bfloat16, device=DEV)
    bep.bep_grouped_gemm_int(ctx, cu, se, codes, scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
    bep.bep_clear_status(ctx)
    assert (y[20:] == 5).all()
    q, wq, ws = codes.cpu().numpy(), w.codes.cpu().numpy(), w.scales.cpu().numpy()
    for a, b, e in ((0, 3, 0), (3, 9, 2), (9, 20, 2)):
        assert np.array_equal(bits(y)[a:b], ref.product_bits(q[a:b], np.ones(b - a, np.float32), wq[e], ws[e]))
    for bad in ([0, 3, 2, 9, 9, 20, 30], [0, 3, 3, 9, 9, 20, 41], [-1, 3, 3, 9, 9, 20, 30]):
        cu[0] = torch.tensor(bad, dtype=torch.int32)
        y.fill_(5.0)
        bep.bep_grouped_gemm_int(ctx, cu, se, codes, scales, w.codes, w.scales, y)
        assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
        bep.bep_clear_status(ctx)
        assert (y == 5).all()
    cu.zero_()   # nothing at all
    bep.bep_grouped_gemm_int(ctx, cu, se, codes, scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0 and (y == 5).all()
    ctx.close()


def test_captured_on_a_side_stream(lib):
    """Dispatch, product, activation and second product in one graph, the contexts' first calls among them."""
    bep = lib
    R, S, E, K, H, F = 2, 24, 8, 2, 128, 64
    up, t = planned(bep, R, S, E, K, H, 2 * F)
    down = bep.Context(bep.Config(R, E, E // R, K, S, F, H, bep.BEP_TRAIN))
    w1, w2 = weights(bep, up), weights(bep, down, 2)
    n = R * S * K
    x = torch.randn(R, S, H, device=DEV).bfloat16()
    r1, r2 = bep.IntRows(n, H), bep.IntRows(n, F)
    h = torch.empty(n, 2 * F, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(n, H, dtype=torch.bfloat16, device=DEV)

    def step():
        bep.bep_dispatch_int(up, x, t["dest"], r1.codes, r1.scales)
        bep.bep_grouped_gemm_int(up, t["cu"], t["se"], r1.codes, r1.scales, w1.codes, w1.scales, h)
        bep.bep_swiglu_int(down, h, r2.codes, r2.scales)
        bep.bep_grouped_gemm_int(down, t["cu"], t["se"], r2.codes, r2.scales, w2.codes, w2.scales, y)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        step()
    outs = []
    for seed in (1, 2):
        x.copy_(torch.randn(R, S, H, device=DEV, generator=torch.Generator(DEV).manual_seed(seed)).bfloat16())
        graph.replay()
        a = y.clone()
        step()
        assert torch.equal(a, y)
        outs.append(a)
    assert not torch.equal(outs[0], outs[1])
    assert bep.bep_status(up) == 0 and bep.bep_status(down) == 0
    up.close()
    down.close()


def test_refusals(lib):
    bep = lib
    ctx, cu, se = one_rank(bep, 8, 128, 64)
    w, r = bep.IntWeight(ctx), bep.IntRows(8, 128)
    x = torch.zeros(1, 8, 128, dtype=torch.bfloat16, device=DEV)
    dest = torch.zeros(1, 8, 1, dtype=torch.int32, device=DEV)
    y = torch.empty(8, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError):
        bep.bep_dispatch_int(ctx, x.float(), dest, r.codes, r.scales)
    with pytest.raises(TypeError):
        bep.bep_dispatch_int(ctx, x, dest, r.codes.view(torch.uint8), r.scales)
    with pytest.raises(ValueError):
        bep.bep_dispatch_int(ctx, x, dest, r.codes[:7], r.scales)
    with pytest.raises(ValueError):
        bep.bep_dispatch_int(ctx, x.cpu(), dest, r.codes, r.scales)
    with pytest.raises(ValueError):
        bep.bep_grouped_gemm_int(ctx, cu, se, r.codes, r.scales, w.codes, w.scales[:, :63], y)
    with pytest.raises(ValueError):
        bep.bep_grouped_gemm_int(ctx, cu, se, r.codes, None, w.codes, w.scales, y)
    with pytest.raises(bep.BepError) as e:   # 96 is no multiple of 64
        bep.bep_swiglu_int(ctx, torch.zeros(8, 192, dtype=torch.bfloat16, device=DEV),
                           torch.zeros(8, 96, dtype=torch.int8, device=DEV), r.scales)
    assert e.value.code == bep.BEP_ERR_ARG
    raw = torch.zeros(8 * 128 + 16, dtype=torch.int8, device=DEV)
    with pytest.raises(bep.BepError) as e:
        bep.bep_dispatch_int(ctx, x, dest, raw[1:1 + 8 * 128].view(8, 128), r.scales)
    assert e.value.code == bep.BEP_ERR_ALIGN
    ctx.close()


def test_calls_without_tokens(lib):
    bep = lib
    ctx = bep.Context(bep.Config(2, 4, 2, 1, 0, 128, 64, bep.BEP_TRAIN))
    L = bep.load()
    assert L.bep_dispatch_int(ctx.handle, None, None, None, None, None) == 0
    assert L.bep_swiglu_int(ctx.handle, None, 64, None, None, None) == 0
    assert L.bep_grouped_gemm_int(ctx.handle, None, None, None, None, None, None, None, None) == 0
    assert bep.bep_status(ctx) == 0
    ctx.close()
