"""Every width of the router's kernels (experts a lane holds), with all lanes full and not: choices, gates,
loads and gradients against the 64-bit reference, gradients with a bound for every entry."""
import numpy as np
import pytest
import torch

import experts_ref as ref
from test_gpu_route import DEV, context, draw_logits, routed, score_tol
from test_gpu_route_gates import dense_bound, gate_bound, gradient, soft_tol

pytestmark = pytest.mark.gpu

# experts a lane holds: 1, 2, 3, 4, 5, 6, 8, 12, 16, 32, 64
WIDTHS = [20, 32, 44, 64, 72, 96, 100, 128, 140, 160, 172, 192, 200, 256, 260, 384, 388, 512, 516, 1024, 1028, 2048]


def drawn(T, E, K, softmax, use_bias, groups, top_groups, group_top, half):
    by_score = use_bias or group_top > 1
    low = ref.LOWEST["bf16" if half else "f32"]
    for seed in range(60):   # inputs without keys nearer than 32 bits can tell apart
        rng = np.random.default_rng([E, K, groups, seed])
        x = draw_logits(rng, T, E, half)
        size = 0.3 / E if softmax else 0.05
        bias = np.float32(rng.normal(size=E) * size).astype(np.float64) if use_bias else None
        want, gap = ref.choose(x, K, softmax, bias, groups, top_groups, group_top, low)
        if gap > 2e-6 * (2.0 / E if softmax and by_score else 1.0):
            return rng, x, bias, want, low
    pytest.fail("no inputs without a near tie")


@pytest.mark.parametrize("half", (False, True))
@pytest.mark.parametrize("softmax", (True, False))
@pytest.mark.parametrize("groups,top_groups,group_top,use_bias", [(1, 1, 1, True), (1, 1, 1, False), (4, 2, 2, True),
                                                                  (4, 2, 2, False), (4, 3, 1, False)])
@pytest.mark.parametrize("E", WIDTHS)
def test_widths(lib, E, groups, top_groups, group_top, use_bias, softmax, half):
    bep = lib
    T, K = 9, min(8, E // 4)
    rng, x, bias, want, low = drawn(T, E, K, softmax, use_bias, groups, top_groups, group_top, half)
    for renorm in (True, False):
        ctx = context(bep, 1, T, E, K)
        rc = bep.RouteConfig(bep.BEP_SCORE_SOFTMAX if softmax else bep.BEP_SCORE_SIGMOID, groups, top_groups,
                             group_top, renorm, 1.5)
        load = torch.zeros(E, dtype=torch.int32, device=DEV)
        lg, topk, g = routed(bep, ctx, rc, x, half, bias, load)
        assert bep.bep_status(ctx) == 0
        assert np.array_equal(topk.cpu().numpy()[0], want)
        assert np.array_equal(load.cpu().numpy(), np.bincount(want.ravel(), minlength=E))
        wg = ref.gates(x, want, softmax, renorm, 1.5, low)
        assert np.all(np.abs(g.cpu().numpy()[0] - wg) <= (soft_tol(E) if softmax else score_tol(E, K)) * wg)
        dg = np.float32(rng.normal(size=(T, K))).astype(np.float64)
        dl = gradient(bep, ctx, rc, lg, topk, dg)
        wd = ref.route_bwd(x, want, dg, softmax, renorm, 1.5, low)
        tol = np.zeros_like(wd)
        if softmax and not renorm:
            tol = dense_bound(x, want, dg, 1.5, E)
        else:
            if softmax:   # the others' gradient is 0: in the reference it cancels to the rounding of 64 bits
                chosen = np.zeros(wd.shape, bool)
                np.put_along_axis(chosen, want, True, 1)
                assert np.all(np.abs(wd[~chosen]) < 1e-14)
                wd = np.where(chosen, wd, 0.0)
            # sigmoid: s (1 - s) a second time around; not renormalised, the dot product is absent
            np.put_along_axis(tol, want, gate_bound(3 * score_tol(K, K), wg / 1.5, dg, 1.5), 1)
        assert np.all(np.abs(dl - wd) <= tol + (2.0 ** -8 * np.abs(wd) if half else 0))
        ctx.close()
