"""4-bit experts on the GPU against the 64-bit reference: codes and scales exactly, products within
the bound of fp32 accumulation and one bf16 rounding."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).bfloat16().to(DEV)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def planned(bep, R, S, E, K, H, Hp, B=None, seed=0, skew=1.0):
    """A context, a routing over skewed experts, and the planner's outputs."""
    mode = bep.BEP_TRAIN if B is None else bep.BEP_INFER
    cfg = bep.Config(R, E, E // R if B is None else B, K, S, H, Hp, mode)
    ctx = bep.Context(cfg)
    p = synth.zipf_popularity(E, skew)
    topk = synth.gumbel_topk(R, S, K, p, seed)
    t = dict(cu=torch.zeros(R, E + cfg.B + 1, dtype=torch.int32, device=DEV),
             se=torch.full((R, cfg.B), -1, dtype=torch.int32, device=DEV),
             dest=torch.zeros(R, S, K, dtype=torch.int32, device=DEV),
             mv=torch.zeros(1, dtype=torch.float64, device=DEV))
    bep.bep_plan(ctx, torch.from_numpy(topk).to(DEV), t["cu"], t["se"], t["dest"], t["mv"])
    assert bep.bep_status(ctx) == 0
    return ctx, t


def row_experts(cfg, t):
    """Expert of every receive row, from the plan's tables (-1: a row of no segment)."""
    cu, se = t["cu"].cpu().numpy(), t["se"].cpu().numpy()
    out = np.full(cfg.R * cfg.C, -1, np.int64)
    for u in range(cfg.R):
        for r in range(cfg.E + cfg.B):
            e = r if r < cfg.E else se[u, r - cfg.E]
            out[u * cfg.C + cu[u, r]:u * cfg.C + cu[u, r + 1]] = e
    return out


def weights(bep, ctx, seed=1):
    c = ctx.cfg
    rng = np.random.default_rng([seed, c.H, c.Hp])
    w = bf16(rng.normal(size=(c.E, c.H, c.Hp)) * 0.02)
    q = bep.MxWeight(ctx)
    bep.bep_mx_quantize_weight(ctx, w, q.codes, q.scales)
    return w, q


def check_product(y, xv, wv, expert, H):
    """y [rows, H'] against fp64 products of the 4-bit values: bf16 rounding and, for each of the
    H / 64 tensor-core steps, a truncated fp32 sum (2^-22 of the magnitudes so far)."""
    for e in np.unique(expert[expert >= 0]):
        at = expert == e
        want = xv[at] @ wv[e].T
        mag = np.abs(xv[at]) @ np.abs(wv[e].T)
        tol = 2.0 ** -8 * np.abs(want) + (H / 64 + 1) * 2.0 ** -22 * mag
        assert np.all(np.abs(y[at] - want) <= tol), f"expert {e}: {np.max(np.abs(y[at] - want) / np.maximum(tol, 1e-30))}"


@pytest.mark.parametrize("E,H,Hp", [(2, 64, 64), (3, 128, 192), (2, 1088, 576), (1, 4160, 128)])
def test_weight_quantisation(lib, E, H, Hp):
    bep = lib
    ctx = bep.Context(bep.Config(1, E, E, 1, 4, H, Hp, bep.BEP_TRAIN))
    rng = np.random.default_rng([E, H])
    v = rng.normal(size=(E, H, Hp)) * np.exp2(rng.integers(-20, 20, size=(E, H // 32, 1, 1))).repeat(32, 1).reshape(E, H, 1)
    v[0, :32, 0] = 0
    v[0, 5, 1] = np.inf
    v[0, 6, 2] = np.nan
    v[0, :32, 3] = 1e-39
    v[0, :32, 4] = 3.3e38
    grid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    v[0, :16, 5] = np.concatenate((grid, -grid))          # ties, largest 6: scale 1
    v[0, 16:32, 5] = 0
    w = bf16(v)
    raw_c = torch.full((E * Hp * H // 2 + 4096,), 0x77, dtype=torch.uint8, device=DEV)
    codes = raw_c[2048:2048 + E * Hp * H // 2].view(E, Hp, H // 2)
    q = bep.MxWeight(ctx)
    bep.bep_mx_quantize_weight(ctx, w, codes, q.scales)
    assert bep.bep_status(ctx) == 0
    assert (raw_c[:2048] == 0x77).all() and (raw_c[-2048:] == 0x77).all()
    wc, wb = ref.mx4(f64(w).transpose(0, 2, 1))
    assert np.array_equal(ref.unblock_scales(q.scales.cpu().numpy(), Hp, H // 32), wb)
    assert np.array_equal(ref.unpack4(codes.cpu().numpy()), wc)
    ctx.close()


@pytest.mark.parametrize("R,S,E,K,H", [(1, 1, 8, 3, 64), (2, 33, 8, 2, 1088), (3, 50, 12, 5, 512), (1, 2, 40, 32, 7168)])
def test_dispatch_in_4_bits(lib, R, S, E, K, H):
    bep = lib
    ctx, t = planned(bep, R, S, E, K, H, 64)
    rng = np.random.default_rng([S, H])
    v = rng.normal(size=(R * S, H)) * np.exp2(rng.integers(-8, 8, size=(R * S, 1)))
    v[0, 0] = np.inf
    v[-1, 32:64] = 0
    x = bf16(v).view(R, S, H)
    rows = bep.MxRows(R * S * K, H)
    rows.scales.fill_(0xEE)
    bep.bep_dispatch_mx(ctx, x, t["dest"], rows.codes, rows.scales)
    assert bep.bep_status(ctx) == 0
    wc, wb = ref.mx4(f64(x).reshape(R * S, H))
    dest = t["dest"].cpu().numpy().reshape(R * S, K)
    codes, sc = ref.unpack4(rows.codes.cpu().numpy()), rows.scales.cpu().numpy()
    for k in range(K):
        assert np.array_equal(codes[dest[:, k]], wc)
        assert np.array_equal(sc[dest[:, k], :H // 32], wb)
    assert np.all(sc[:, H // 32:] == 0xEE)
    ctx.close()


def test_dispatch_skips_bad_destinations(lib):
    bep = lib
    ctx, t = planned(bep, 2, 16, 8, 2, 128, 64)
    dest = t["dest"].clone()
    dest[0, 3, 1], dest[1, 0, 0] = 64, -1
    raw = torch.full((64 * 64 + 8192,), 0x33, dtype=torch.uint8, device=DEV)
    rows = bep.MxRows(64, 128)
    bep.bep_dispatch_mx(ctx, torch.ones(2, 16, 128, dtype=torch.bfloat16, device=DEV), dest,
                        raw[4096:4096 + 64 * 64].view(64, 64), rows.scales)
    assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
    assert (raw[:4096] == 0x33).all() and (raw[-4096:] == 0x33).all()
    ctx.close()


@pytest.mark.parametrize("rows,F", [(1, 64), (37, 1088), (300, 512), (5, 8192)])
def test_activation_in_4_bits(lib, rows, F):
    bep = lib
    ctx = bep.Context(bep.Config(1, 1, 1, 1, rows, 64, 64, bep.BEP_TRAIN))
    rng = np.random.default_rng([rows, F])
    h = bf16(rng.normal(size=(rows, 2 * F)) * 2)
    q = bep.MxRows(rows, F)
    bep.bep_swiglu_mx(ctx, h, q.codes, q.scales)
    assert bep.bep_status(ctx) == 0
    a = ref.swiglu(f64(h))
    wc, wb = ref.mx4(a)
    got, sc = ref.unpack4(q.codes.cpu().numpy()), q.scales.cpu().numpy()[:, :F // 32]
    # a value within 2^-18 of a rounding boundary may go to either side; nothing else may differ
    b = a.reshape(rows, -1, 32)
    near_scale = np.abs(np.log2(np.abs(b).max(-1) / 6.0) % 1.0) < 1e-5
    assert np.all((sc == wb) | near_scale)
    v = np.abs(np.ldexp(b, -(wb[..., None].astype(np.int64) - 127)))
    mids = (ref.E2M1[1:] + ref.E2M1[:-1]) / 2
    near = (np.abs(v[..., None] - mids) < 2.0 ** -17 * mids).any(-1) | near_scale[..., None]
    tiny = (wc & 7) == 0                       # the sign of a zero that underflowed may differ
    same = (got == wc) | (tiny & ((got & 7) == 0))
    assert np.all(same | near.reshape(rows, F))
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
]


@pytest.mark.parametrize("R,S,E,K,H,Hp,B,skew", PRODUCTS)
def test_product(lib, R, S, E, K, H, Hp, B, skew):
    bep = lib
    ctx, t = planned(bep, R, S, E, K, H, Hp, B, seed=3, skew=skew)
    c = ctx.cfg
    _, w = weights(bep, ctx)
    rng = np.random.default_rng([R, S, H])
    x = bf16(rng.normal(size=(R, S, H)))
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
    # the same call again gives the same bits
    y2 = torch.empty_like(y)
    bep.bep_grouped_gemm_mx(ctx, t["cu"], t["se"], rows.codes, rows.scales, w.codes, w.scales, y2)
    assert torch.equal(y2.view(torch.int16), y.view(torch.int16))
    ctx.close()


def test_each_element_and_scale_has_its_place(lib):
    """One-hot rows with a scale of their own against weights that are different at every position."""
    bep = lib
    H, Hp, E = 320, 192, 2
    rows_n = H
    ctx = bep.Context(bep.Config(1, E, E, 1, rows_n, H, Hp, bep.BEP_TRAIN))
    rng = np.random.default_rng(0)
    wv = rng.choice(np.array([0.5, 1, 1.5, 2, 3, 4, 6, -1, -3, -6]), size=(E, H, Hp))
    wv *= np.exp2(rng.integers(-9, 9, size=(E, H // 32, Hp))).repeat(32, 1)
    w = bep.MxWeight(ctx)
    bep.bep_mx_quantize_weight(ctx, bf16(wv), w.codes, w.scales)
    got = ref.mx4_values(ref.unpack4(w.codes.cpu().numpy()), ref.unblock_scales(w.scales.cpu().numpy(), Hp, H // 32))
    x = np.zeros((rows_n, H))
    x[np.arange(rows_n), np.arange(rows_n)] = np.exp2(np.arange(rows_n) % 11 - 5) * 3
    rows = bep.MxRows(rows_n, H)
    dest = torch.arange(rows_n, dtype=torch.int32, device=DEV).view(1, rows_n, 1)
    bep.bep_dispatch_mx(ctx, bf16(x).view(1, rows_n, H), dest, rows.codes, rows.scales)
    cu = torch.tensor([[0, 150, rows_n, rows_n, rows_n]], dtype=torch.int32, device=DEV)
    y = torch.empty(rows_n, Hp, dtype=torch.bfloat16, device=DEV)
    se = torch.full((1, E), -1, dtype=torch.int32, device=DEV)
    bep.bep_grouped_gemm_mx(ctx, cu, se, rows.codes, rows.scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0
    want = np.concatenate((x[:150] @ got[0].T, x[150:] @ got[1].T))
    # one product a sum, of two values of 2 significant bits: exact in bf16
    assert np.array_equal(f64(y), want)
    ctx.close()


def test_nan_blocks_stay_in_their_rows_and_columns(lib):
    bep = lib
    H, Hp, n = 256, 128, 40
    ctx = bep.Context(bep.Config(1, 1, 1, 1, n, H, Hp, bep.BEP_TRAIN))
    rng = np.random.default_rng(2)
    x = rng.normal(size=(n, H))
    x[17, 100] = np.inf
    wv = rng.normal(size=(1, H, Hp))
    wv[0, 200, 33] = np.nan
    w = bep.MxWeight(ctx)
    bep.bep_mx_quantize_weight(ctx, bf16(wv), w.codes, w.scales)
    rows = bep.MxRows(n, H)
    dest = torch.arange(n, dtype=torch.int32, device=DEV).view(1, n, 1)
    bep.bep_dispatch_mx(ctx, bf16(x).view(1, n, H), dest, rows.codes, rows.scales)
    cu = torch.tensor([[0, n, n]], dtype=torch.int32, device=DEV)
    y = torch.empty(n, Hp, dtype=torch.bfloat16, device=DEV)
    bep.bep_grouped_gemm_mx(ctx, cu, torch.full((1, 1), -1, dtype=torch.int32, device=DEV), rows.codes, rows.scales,
                            w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0
    nan = np.isnan(f64(y))
    want = np.zeros((n, Hp), bool)
    want[17, :] = True
    want[:, 33] = True
    assert np.array_equal(nan, want)
    ctx.close()


def test_bad_tables(lib):
    bep = lib
    ctx, t = planned(bep, 2, 64, 8, 2, 128, 64, None, skew=1.2)
    _, w = weights(bep, ctx)
    rows = bep.MxRows(256, 128)
    bep.bep_dispatch_mx(ctx, torch.ones(2, 64, 128, dtype=torch.bfloat16, device=DEV), t["dest"], rows.codes, rows.scales)
    raw = torch.full((256 * 64 + 8192,), 9.0, dtype=torch.bfloat16, device=DEV)
    y = raw[4096:4096 + 256 * 64].view(256, 64)
    cu = t["cu"].clone()
    cu[1, 3] = cu[1, 4] + 1
    bep.bep_grouped_gemm_mx(ctx, cu, t["se"], rows.codes, rows.scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS and (raw == 9).all()
    bep.bep_clear_status(ctx)
    # a slot segment whose expert is unknown is skipped, the others are computed
    cu = torch.zeros_like(t["cu"])
    cu[0, 9:] = 100
    cu[1, 1:] = 128
    for bad in (-1, 8):
        se = torch.full_like(t["se"], bad)
        raw.fill_(9.0)
        bep.bep_grouped_gemm_mx(ctx, cu, se, rows.codes, rows.scales, w.codes, w.scales, y)
        assert bep.bep_status(ctx) == bep.BEP_DERR_BOUNDS
        assert (y[:128] == 9).all() and not (y[128:] == 9).all(1).any()
        assert (raw[:4096] == 9).all() and (raw[-4096:] == 9).all()
        bep.bep_clear_status(ctx)
    # rows outside every segment are not written
    cu.zero_()
    cu[0, 1:] = 37
    raw.fill_(9.0)
    bep.bep_grouped_gemm_mx(ctx, cu, t["se"], rows.codes, rows.scales, w.codes, w.scales, y)
    assert bep.bep_status(ctx) == 0
    assert (y[37:] == 9).all() and not (y[:37] == 9).all(1).any()
    ctx.close()


def test_another_stream_no_rows_and_refusals(lib):
    bep = lib
    ctx, t = planned(bep, 2, 64, 8, 2, 256, 128, None)
    _, w = weights(bep, ctx)
    rows = bep.MxRows(256, 256)
    x = torch.randn(2, 64, 256, device=DEV).bfloat16()
    y = [torch.empty(256, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for out, stream in zip(y, (None, st)):
        bep.bep_dispatch_mx(ctx, x, t["dest"], rows.codes, rows.scales, stream=stream)
        bep.bep_grouped_gemm_mx(ctx, t["cu"], t["se"], rows.codes, rows.scales, w.codes, w.scales, out, stream=stream)
        torch.cuda.synchronize()
    assert torch.equal(*y)
    with pytest.raises(TypeError):
        bep.bep_dispatch_mx(ctx, x.float(), t["dest"], rows.codes, rows.scales)
    with pytest.raises(ValueError):
        bep.bep_dispatch_mx(ctx, x, t["dest"], rows.codes, rows.scales[:, :8])
    with pytest.raises(ValueError):
        bep.bep_dispatch_mx(ctx, x.transpose(0, 1), t["dest"], rows.codes, rows.scales)
    with pytest.raises(ValueError):
        bep.bep_grouped_gemm_mx(ctx, t["cu"], t["se"], rows.codes, rows.scales, w.codes[:1], w.scales, y[0])
    with pytest.raises(TypeError):
        bep.bep_grouped_gemm_mx(ctx, t["cu"], t["se"], rows.codes, rows.scales, w.codes, w.scales, y[0].float())
    h = torch.randn(256, 2 * 96, device=DEV).bfloat16()
    with pytest.raises(bep.BepError) as e:      # F = 96 is not a multiple of 64
        bep.bep_swiglu_mx(ctx, h, torch.empty(256, 48, dtype=torch.uint8, device=DEV), rows.scales)
    assert e.value.code == bep.BEP_ERR_ARG
    off = torch.empty(256 * 128 + 16, dtype=torch.uint8, device=DEV)[1:1 + 256 * 128].view(256, 128)
    with pytest.raises(bep.BepError) as e:
        bep.bep_dispatch_mx(ctx, x, t["dest"], off, rows.scales)
    assert e.value.code == bep.BEP_ERR_ALIGN
    assert bep.bep_status(ctx) == 0
    ctx.close()
    ctx = bep.Context(bep.Config(2, 8, 4, 2, 0, 256, 128, bep.BEP_TRAIN))
    cu = torch.zeros(2, 13, dtype=torch.int32, device=DEV)
    e = torch.empty(0, dtype=torch.uint8, device=DEV)
    bep.bep_grouped_gemm_mx(ctx, cu, t["se"], e, e, w.codes, w.scales, y[0][:0])
    assert bep.bep_status(ctx) == 0
    ctx.close()


@pytest.mark.parametrize("R,S,E,K,H,Hp", [(8, 61, 24, 4, 7168, 256), (2, 900, 4, 2, 256, 1344), (1, 2000, 3, 1, 512, 192)])
def test_calls_in_a_row_give_the_same_bits(lib, R, S, E, K, H, Hp):
    """Dispatch and product queued many times without a wait between them: launches overlap, rings and
    accumulators wrap, and rows are rewritten while the call before has just ended."""
    bep = lib
    ctx, t = planned(bep, R, S, E, K, H, Hp, None, seed=5, skew=1.0)
    _, w = weights(bep, ctx)
    x = [torch.randn(R, S, H, device=DEV).bfloat16() for _ in range(2)]
    rows = bep.MxRows(R * S * K, H)
    y = [torch.empty(R * S * K, Hp, dtype=torch.bfloat16, device=DEV) for _ in range(12)]
    for i, out in enumerate(y):
        bep.bep_dispatch_mx(ctx, x[i % 2], t["dest"], rows.codes, rows.scales)
        bep.bep_grouped_gemm_mx(ctx, t["cu"], t["se"], rows.codes, rows.scales, w.codes, w.scales, out)
    assert bep.bep_status(ctx) == 0
    for i in range(2, 12):
        assert torch.equal(y[i].view(torch.int16), y[i % 2].view(torch.int16))
    assert not torch.equal(y[0], y[1])
    ctx.close()


def test_a_graph_and_an_sm_budget_give_the_same_bits(lib):
    bep = lib
    ctx, t = planned(bep, 4, 300, 16, 3, 576, 320, None, skew=1.0)
    _, w = weights(bep, ctx)
    x = torch.randn(4, 300, 576, device=DEV).bfloat16()
    rows, y = bep.MxRows(3600, 576), torch.empty(3600, 320, dtype=torch.bfloat16, device=DEV)

    def step():
        bep.bep_dispatch_mx(ctx, x, t["dest"], rows.codes, rows.scales)
        bep.bep_grouped_gemm_mx(ctx, t["cu"], t["se"], rows.codes, rows.scales, w.codes, w.scales, y)

    step()
    torch.cuda.synchronize()
    want = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
        step()
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    bep.bep_set_comm_sms(ctx, 3)
    y.zero_()
    step()
    assert bep.bep_status(ctx) == 0
    assert torch.equal(y, want)
    ctx.close()
