"""Gates and logit gradients of the router where scores lie far apart, against the 64-bit reference, with
a bound for every entry from its own terms."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from test_gpu_route import DEV, context, routed, score_tol

pytestmark = pytest.mark.gpu
LOW = ref.LOWEST["f32"]


def gradient(bep, ctx, rc, lg, topk, dg):
    dl = torch.full_like(lg, float("nan"))
    bep.bep_route_bwd(ctx, rc, lg, topk, torch.from_numpy(np.float32(dg)).to(DEV).view(topk.shape), dl)
    return dl.float().cpu().numpy().reshape(-1, ctx.cfg.E).astype(np.float64)


def gate_bound(rel, w, dg, scale):
    """|error| of scale * w_k (dg_k - sum_j dg_j w_j): each factor has a relative error below rel."""
    return rel * scale * w * (np.abs(dg) + (np.abs(dg) * w).sum(1, keepdims=True))


@pytest.mark.parametrize("E,K", [(8, 3), (64, 4), (90, 5), (384, 8)])
@pytest.mark.parametrize("off", (-np.inf, -1e9))
def test_renormalised_gates_without_the_dominant_expert(lib, E, K, off):
    """A bias disables the expert whose logit leads by d: the others' gates do not depend on d."""
    bep = lib
    lead = np.array([0.0, 20.0, 60.0, 85.0, 88.0, 95.0, 100.0, 104.0, 150.0, 600.0])
    T = len(lead)
    x = np.tile(-0.375 * np.minimum(np.arange(E), 24.0), (T, 1))   # falls with e, as the bias does
    x[:, 2] = lead + 5
    bias = np.float32(0.01 * (E - np.arange(E))).astype(np.float64)
    bias[2] = off
    want = np.tile(np.r_[0, 1, 3:K + 1], (T, 1))
    ctx = context(bep, 1, T, E, K)
    rc = bep.RouteConfig(bep.BEP_SCORE_SOFTMAX, renorm=True, scale=2.5)
    lg, topk, g = routed(bep, ctx, rc, x, False, bias)
    assert bep.bep_status(ctx) == 0
    assert np.array_equal(topk.cpu().numpy()[0], want)
    w = np.exp(np.take_along_axis(x, want, 1))
    w /= w.sum(1, keepdims=True)
    got = g.cpu().numpy()[0].astype(np.float64)
    assert np.all(np.abs(got - 2.5 * w) <= score_tol(K, K) * 2.5 * w)
    dg = np.float32(np.random.default_rng([E, K]).normal(size=(T, K))).astype(np.float64)
    dl = gradient(bep, ctx, rc, lg, topk, dg)
    wd = ref.route_bwd(x, want, dg, True, True, 2.5, LOW)
    tol = np.zeros_like(wd)
    np.put_along_axis(tol, want, gate_bound(2 * score_tol(K, K), w, dg, 2.5), 1)
    # the reference's own row sum cancels to 1e-16 of the largest term, which the dominant score scales
    s, _ = ref.scores(x, True, LOW)
    assert np.all(np.abs(dl - wd) <= tol + 1e-14 * s)
    ctx.close()


# Relative error of a softmax gate, in units of 2^-24: expf 4 and the row's exponentials 4 (2 units in the
# last place each) and up to 6 from their arguments (x - top) log2(e), rounded at magnitudes of 8 here; the
# sum of E terms, lane by lane and over 5 butterfly steps; the reciprocal, two products and the scale, 4.
def soft_tol(E):
    return (4 + 4 + 6 + E / 32 + 5 + 4) * 2.0 ** -24


def fast_rel(x, E):
    """The same for the score of any expert: its own argument is rounded relative to its distance from the
    row's largest logit (1.5 roundings of it, the constant's one among them)."""
    return soft_tol(E) + (x.max(1, keepdims=True) - x) * 2.0 ** -23


def dense_bound(x, topk, dg, scale, E):
    """|error| of scale * s_e (dg_e - sum_k dg_k s_k), dg_e = 0 for the others, from its own terms."""
    s, _ = ref.scores(x, True, LOW)
    rel = fast_rel(x, E)
    at = np.zeros_like(s)
    np.put_along_axis(at, topk, np.abs(dg), 1)
    return 2 * scale * rel * s * (at + (at * s).sum(1, keepdims=True))


@pytest.mark.parametrize("E,K", [(8, 2), (33, 7), (128, 8), (192, 6), (384, 8), (512, 16), (2048, 32)])
@pytest.mark.parametrize("off", (0.0, 30.0, -30.0, 37.0, -37.0, 500.0))
@pytest.mark.parametrize("use_bias", (False, True))
def test_softmax_gates_and_every_gradient(lib, E, K, off, use_bias):
    """Gates that are not renormalised, and the gradient of every logit, around a common offset."""
    bep = lib
    T = 24
    for seed in range(40):
        rng = np.random.default_rng([E, K, seed])
        x = np.clip(np.round(rng.normal(size=(T, E)) * 1.0 * 4096) / 4096, -2.75, 2.75) + off
        bias = np.float32(rng.normal(size=E) * 0.3 / E).astype(np.float64) if use_bias else None
        want, gap = ref.choose(x, K, True, bias, 1, 1, 1, LOW)
        if gap > 4e-6 / E:
            break
    else:
        pytest.fail("no inputs without a near tie")
    ctx = context(bep, 1, T, E, K)
    rc = bep.RouteConfig(bep.BEP_SCORE_SOFTMAX, renorm=False, scale=1.5)
    lg, topk, g = routed(bep, ctx, rc, x, False, bias)
    assert bep.bep_status(ctx) == 0
    assert np.array_equal(topk.cpu().numpy()[0], want)
    wg = ref.gates(x, want, True, False, 1.5, LOW)
    assert np.all(np.abs(g.cpu().numpy()[0] - wg) <= soft_tol(E) * wg)
    dg = np.float32(rng.normal(size=(T, K))).astype(np.float64)
    dl = gradient(bep, ctx, rc, lg, topk, dg)
    wd = ref.route_bwd(x, want, dg, True, False, 1.5, LOW)
    assert np.all(np.abs(dl - wd) <= dense_bound(x, want, dg, 1.5, E))
    ctx.close()


@pytest.mark.parametrize("E,K", [(8, 3), (64, 4), (90, 5), (384, 8), (2048, 32)])
@pytest.mark.parametrize("softmax", (False, True))
@pytest.mark.parametrize("groups", (1, 2))
@pytest.mark.parametrize("renorm", (True, False))
def test_scores_below_the_smallest_normal(lib, E, K, softmax, groups, renorm):
    """Scores that fp32 holds as subnormals only: still in order, and renormalised gates keep their ratios."""
    bep = lib
    x = np.full((3, E), -102.0)
    # the best have the highest indices, a quarter apart: their scores differ by 20 units of 2^-149 or more
    x[:, E - K:] = -(88.0 + 12.0 / (K + 1) * np.arange(1, K + 1))[::-1] + np.zeros((3, 1))
    if softmax:
        x[:, 0] = 0.0                             # the row's largest, and the first choice
        x[1, 0] = 10.0
        x[1, 1:] += 10.0
    if groups == 2 and softmax:
        x[:, E // 2] = x[:, 0]                    # in the group of the others
        x[:, 0] = -102.0
    x = np.float32(x).astype(np.float64)
    bias = np.zeros(E) if groups == 1 else None   # groups of two keys: by score without a bias
    want, _ = ref.choose(x, K, softmax, bias, groups, 1, 2 if groups > 1 else 1, LOW)
    ctx = context(bep, 1, 3, E, K)
    rc = bep.RouteConfig(bep.BEP_SCORE_SOFTMAX if softmax else bep.BEP_SCORE_SIGMOID, groups=groups, top_groups=1,
                         group_top=2 if groups > 1 else 1, renorm=renorm, scale=2.0)
    lg, topk, g = routed(bep, ctx, rc, x, False, bias)
    assert bep.bep_status(ctx) == 0
    assert np.array_equal(topk.cpu().numpy()[0], want)
    wg = ref.gates(x, want, softmax, renorm, 2.0, LOW)
    # half a unit of a subnormal score or gate, and the scale; normal ones within a few roundings
    assert np.all(np.abs(g.cpu().numpy()[0] - wg) <= soft_tol(E) * wg + 4 * 2.0 ** -149)
    if renorm and not softmax:
        dg = np.float32(np.random.default_rng(E).normal(size=(3, K))).astype(np.float64)
        dl = gradient(bep, ctx, rc, lg, topk, dg)
        wd = ref.route_bwd(x, want, dg, False, True, 2.0, LOW)
        tol = np.zeros_like(wd)
        np.put_along_axis(tol, want, gate_bound(2 * score_tol(K, K), wg / 2, dg, 2.0), 1)
        assert np.all(np.abs(dl - wd) <= tol)
    ctx.close()
