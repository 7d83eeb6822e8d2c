"""Routing on the GPU against the 64-bit reference: choices exactly, gates and gradients within
the rounding of 32-bit arithmetic."""
import numpy as np
import pytest
import torch

import experts_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def context(bep, R, S, E, K):
    return bep.Context(bep.Config(R, E, E // R, K, S, 64, 64, bep.BEP_TRAIN))


def draw_logits(rng, T, E, half):
    x = rng.normal(size=(T, E)) * 1.5
    # a grid (exact in bf16 and fp32) with many equal logits
    return np.round(x * 16) / 16 if half else np.round(x * 4096) / 4096


def routed(bep, ctx, rc, x, half, bias=None, load=None, R=None, stream=None):
    c = ctx.cfg
    lg = torch.from_numpy(np.asarray(x, np.float32)).to(DEV).view(c.R, c.S, c.E)
    if half:
        lg = lg.bfloat16()
    topk = torch.full((c.R, c.S, c.K), -7, dtype=torch.int32, device=DEV)
    g = torch.full((c.R, c.S, c.K), float("nan"), device=DEV)
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).to(DEV)
    bep.bep_route(ctx, rc, lg, topk, g, bias=b, load=load, stream=stream)
    return lg, topk, g


# fp32 error of a score: expf and a division (each 2 units or fewer) and a sum of E terms, lane
# by lane (E/32) and over 5 butterfly steps
def score_tol(E, K):
    return (E / 32 + 5 + K + 12) * 2.0 ** -24


CASES = [
    # R, S, E, K, softmax, groups, top_groups, group_top, bias, renorm, scale
    (1, 1, 1, 1, True, 1, 1, 1, False, True, 1.0),
    (1, 1, 8, 8, False, 1, 1, 1, True, True, 2.5),
    (2, 64, 8, 2, True, 1, 1, 1, False, True, 1.0),
    (8, 1, 384, 8, False, 8, 4, 2, True, True, 2.5),
    (3, 37, 90, 5, True, 6, 3, 1, False, False, 1.0),
    (3, 37, 90, 5, False, 6, 2, 2, False, True, 1.0),
    (1, 70, 33, 7, True, 1, 1, 1, True, False, 0.5),
    (1, 19, 33, 32, False, 3, 3, 1, False, False, 1.0),
    (2, 31, 130, 1, True, 13, 2, 2, True, True, 1.0),
    (1, 50, 256, 8, False, 32, 9, 2, True, False, 1.0),
    (1, 40, 512, 16, True, 16, 5, 2, False, False, 3.0),
    (1, 9, 1000, 12, False, 1, 1, 1, False, True, 1.0),
    (1, 7, 2048, 32, True, 8, 3, 2, True, True, 1.0),
]


@pytest.mark.parametrize("half", (False, True))
@pytest.mark.parametrize("case", CASES)
def test_route_and_gradient(lib, case, half):
    bep = lib
    R, S, E, K, softmax, groups, top_groups, group_top, use_bias, renorm, scale = case
    T = R * S
    low = ref.LOWEST["bf16" if half else "f32"]
    for seed in range(20):   # inputs without keys nearer than 32 bits can tell apart
        rng = np.random.default_rng([E, K, T, seed])
        x = draw_logits(rng, T, E, half)
        bias = np.float32(rng.normal(size=E) * (0.3 / E if softmax else 0.05)).astype(np.float64) if use_bias else None
        want, gap = ref.choose(x, K, softmax, bias, groups, top_groups, group_top, low)
        if gap > 1e-6 * (2.0 / E if softmax and (use_bias or group_top > 1) else 1.0) * 2:
            break
    else:
        pytest.fail("no inputs without a near tie")
    ctx = context(bep, R, S, E, K)
    rc = bep.RouteConfig(bep.BEP_SCORE_SOFTMAX if softmax else bep.BEP_SCORE_SIGMOID, groups, top_groups,
                         group_top, renorm, scale)
    load = torch.full((E,), 3, dtype=torch.int32, device=DEV)
    lg, topk, g = routed(bep, ctx, rc, x, half, bias, load)
    assert bep.bep_status(ctx) == 0
    assert np.array_equal(topk.cpu().numpy().reshape(T, K), want)
    wg = ref.gates(x, want, softmax, renorm, scale, low)
    got = g.cpu().numpy().reshape(T, K).astype(np.float64)
    assert np.all(np.abs(got - wg) <= score_tol(E, K) * np.abs(wg) + 1e-30)
    assert np.array_equal(load.cpu().numpy(), 3 + np.bincount(want.ravel(), minlength=E))
    dg = np.float32(rng.normal(size=(T, K)))
    dl = torch.full_like(lg, float("nan"))
    bep.bep_route_bwd(ctx, rc, lg, topk, torch.from_numpy(dg).to(DEV).view(R, S, K), dl)
    assert bep.bep_status(ctx) == 0
    wd = ref.route_bwd(x, want, dg.astype(np.float64), softmax, renorm, scale, low)
    # dv_k - sum cancels: the error scales with the largest |dg| of the token and with s
    big = scale * np.abs(dg).max(1, keepdims=True) * (1.0 if renorm or not softmax else 2.0)
    tol = 4 * score_tol(E, K) * big * K + (2.0 ** -8 * np.abs(wd) if half else 0)
    assert np.all(np.abs(dl.float().cpu().numpy().reshape(T, E) - wd) <= tol)
    ctx.close()


def test_masks_and_rows_without_experts(lib):
    bep = lib
    E, K, S = 48, 4, 6
    for half in (False, True):
        low = ref.LOWEST["bf16" if half else "f32"]
        for softmax in (True, False):
            for renorm in (True, False):
                rng = np.random.default_rng(3)
                x = draw_logits(rng, S, E, True)
                x[0] = -np.inf                       # nothing left
                x[1] = low                           # the same by the type's lowest value
                x[2, 5:] = -np.inf                   # 5 experts
                x[3, 2:] = low                       # 2 experts: masked ones fill the choice
                x[4, :40] = -np.inf                  # a group left
                bias = np.full(E, 0.01)
                ctx = context(bep, 1, S, E, K)
                rc = bep.RouteConfig(bep.BEP_SCORE_SOFTMAX if softmax else bep.BEP_SCORE_SIGMOID, 6, 3, 2,
                                     renorm, 1.0)
                lg, topk, g = routed(bep, ctx, rc, x, half, bias)
                assert bep.bep_status(ctx) == 0
                want, _ = ref.choose(x, K, softmax, np.float32(bias).astype(float), 6, 3, 2, low)
                assert np.array_equal(topk.cpu().numpy()[0], want)
                wg = ref.gates(x, want, softmax, renorm, 1.0, low)
                got = g.cpu().numpy()[0]
                assert np.all(np.abs(got - wg) <= score_tol(E, K) * wg)
                assert np.all(got[0] == 0) and np.all(got[1] == 0) and np.all(got[3, 2:] == 0)
                dl = torch.full_like(lg, float("nan"))
                dg = torch.ones(1, S, K, device=DEV) * torch.arange(1, K + 1, device=DEV)
                bep.bep_route_bwd(ctx, rc, lg, topk, dg, dl)
                d = dl.float().cpu().numpy()[0]
                wd = ref.route_bwd(x, want, dg.cpu().numpy()[0].astype(float), softmax, renorm, 1.0, low)
                assert np.all(np.isfinite(d))
                assert np.all(np.abs(d - wd) <= 16 * K * score_tol(E, K) + 2.0 ** -8 * np.abs(wd))
                assert np.all(d[0] == 0) and np.all(d[2, 5:] == 0)
                ctx.close()


def test_nonfinite_logits_are_reported(lib):
    bep = lib
    E, K = 40, 3
    for bad in (float("nan"), float("inf")):
        ctx = context(bep, 1, 2, E, K)
        x = np.tile(np.arange(E, dtype=float), (2, 1))
        x[1, 39] = bad
        rc = bep.RouteConfig(renorm=True)
        _, topk, g = routed(bep, ctx, rc, x, False)
        assert bep.bep_status(ctx) == bep.BEP_DERR_NONFINITE
        assert topk.cpu().tolist()[0] == [[39, 38, 37], [38, 37, 36]]
        assert torch.isfinite(g).all()
        bep.bep_clear_status(ctx)
        ctx.close()


def test_extreme_finite_logits(lib):
    bep = lib
    E, K = 64, 4
    x = np.zeros((3, E))
    x[0, 7] = 3e38
    x[1, :] = -3e38
    x[1, 9] = -2.9e38
    x[2, ::2] = 88.0
    for softmax in (True, False):
        ctx = context(bep, 1, 3, E, K)
        rc = bep.RouteConfig(bep.BEP_SCORE_SOFTMAX if softmax else bep.BEP_SCORE_SIGMOID, renorm=True)
        lg, topk, g = routed(bep, ctx, rc, x, False)
        assert bep.bep_status(ctx) == 0
        x32 = x.astype(np.float32).astype(float)
        want, _ = ref.choose(x32, K, softmax, None, 1, 1, 1, ref.LOWEST["f32"])
        assert np.array_equal(topk.cpu().numpy()[0], want)
        assert torch.isfinite(g).all()
        dl = torch.empty_like(lg)
        bep.bep_route_bwd(ctx, rc, lg, topk, torch.ones(1, 3, K, device=DEV), dl)
        assert torch.isfinite(dl).all()
        ctx.close()


def test_bad_choice_in_backward_is_skipped(lib):
    bep = lib
    ctx = context(bep, 1, 4, 24, 3)
    lg = torch.randn(1, 4, 24, device=DEV)
    topk = torch.tensor([[[0, 1, 2], [3, 24, 5], [-1, 4, 6], [7, 8, 9]]], dtype=torch.int32, device=DEV)
    for renorm in (True, False):
        raw = torch.full((4 * 24 + 512,), 5.0, device=DEV)
        dl = raw[256:256 + 96].view(1, 4, 24)
        bep.bep_route_bwd(ctx, bep.RouteConfig(renorm=renorm), lg, topk, torch.ones(1, 4, 3, device=DEV), dl)
        assert bep.bep_status(ctx) == bep.BEP_DERR_EXPERT_ID
        assert (raw[:256] == 5).all() and (raw[-256:] == 5).all()
        bep.bep_clear_status(ctx)
    ctx.close()


def test_another_stream_and_no_tokens(lib):
    bep = lib
    E, K, S = 64, 4, 2000
    ctx = context(bep, 4, S, E, K)
    x = draw_logits(np.random.default_rng(1), 4 * S, E, True)
    rc = bep.RouteConfig()
    _, a, ga = routed(bep, ctx, rc, x, False)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        _, b, gb = routed(bep, ctx, rc, x, False, stream=st)
    st.synchronize()
    assert torch.equal(a, b) and torch.equal(ga, gb)
    ctx.close()
    ctx = context(bep, 4, 0, E, K)
    e = torch.empty(0, device=DEV)
    bep.bep_route(ctx, rc, e, e.int(), e)
    bep.bep_route_bwd(ctx, rc, e, e.int(), e, e)
    assert bep.bep_status(ctx) == 0
    ctx.close()


def test_refusals(lib):
    bep = lib
    R, S, E, K = 2, 4, 24, 3
    ctx = context(bep, R, S, E, K)
    lg = torch.randn(R, S, E, device=DEV)
    topk = torch.empty(R, S, K, dtype=torch.int32, device=DEV)
    g = torch.empty(R, S, K, device=DEV)

    def code(**kw):
        with pytest.raises(bep.BepError) as err:
            bep.bep_route(ctx, bep.RouteConfig(**kw), lg, topk, g)
        return err.value.code

    assert code(score=2) == bep.BEP_ERR_ARG
    assert code(groups=0) == bep.BEP_ERR_ARG
    assert code(groups=4, top_groups=5) == bep.BEP_ERR_ARG
    assert code(groups=4, top_groups=0) == bep.BEP_ERR_ARG
    assert code(groups=4, top_groups=2, group_top=3) == bep.BEP_ERR_ARG
    assert code(scale=float("inf")) == bep.BEP_ERR_ARG
    assert code(groups=5) == bep.BEP_ERR_SIZE
    assert code(groups=12, top_groups=1) == bep.BEP_ERR_SIZE   # 2 experts for K = 3
    rc = bep.RouteConfig()
    with pytest.raises(TypeError):
        bep.bep_route(ctx, rc, lg.half(), topk, g)
    with pytest.raises(TypeError):
        bep.bep_route(ctx, rc, lg, topk.long(), g)
    with pytest.raises(ValueError):
        bep.bep_route(ctx, rc, lg[:, :, :12], topk, g)
    with pytest.raises(ValueError):
        bep.bep_route(ctx, rc, lg.transpose(1, 2).contiguous().transpose(1, 2), topk, g)
    with pytest.raises(ValueError):
        bep.bep_route(ctx, rc, lg.cpu(), topk, g)
    with pytest.raises(ValueError):
        bep.bep_route(ctx, rc, lg, topk, g, bias=torch.zeros(E + 1, device=DEV))
    with pytest.raises(TypeError):
        bep.bep_route_bwd(ctx, rc, lg, topk, g, torch.empty_like(lg, dtype=torch.bfloat16))
    with pytest.raises(bep.BepError):
        bep.bep_route_bwd(ctx, rc, lg, topk, g, lg)
    assert bep.bep_status(ctx) == 0
    ctx.close()


@pytest.mark.parametrize("E,K", [(64, 4), (384, 8), (90, 3)])
def test_negative_and_mixed_keys(lib, E, K):
    """Biases that leave no key, a few, or K keys positive."""
    bep = lib
    S = 40
    for softmax in (True, False):
        for shift in (-2.0, -0.5, -0.02, 0.0):
            for seed in range(20):
                rng = np.random.default_rng([E, seed, int(-100 * shift)])
                x = draw_logits(rng, S, E, False)
                bias = np.float32(rng.normal(size=E) * 0.05 + shift).astype(np.float64)
                want, gap = ref.choose(x, K, softmax, bias, 1, 1, 1, ref.LOWEST["f32"])
                if gap > 4e-6:
                    break
            else:
                pytest.fail("no inputs without a near tie")
            ctx = context(bep, 1, S, E, K)
            rc = bep.RouteConfig(bep.BEP_SCORE_SOFTMAX if softmax else bep.BEP_SCORE_SIGMOID)
            _, topk, g = routed(bep, ctx, rc, x, False, bias)
            assert bep.bep_status(ctx) == 0
            assert np.array_equal(topk.cpu().numpy()[0], want)
            assert np.all(np.abs(g.cpu().numpy()[0] - ref.gates(x, want, softmax, True, 1.0, ref.LOWEST["f32"]))
                          <= score_tol(E, K))
            ctx.close()
    # equal keys, positive and negative, across lanes and registers: the lowest experts
    for shift in (-3.0, 3.0):
        ctx = context(bep, 1, 1, E, K)
        _, topk, _ = routed(bep, ctx, bep.RouteConfig(bep.BEP_SCORE_SIGMOID), np.zeros((1, E)), False,
                            np.full(E, shift))
        assert topk.cpu().tolist()[0][0] == list(range(K))
        ctx.close()
