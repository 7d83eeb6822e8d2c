"""The 64-bit references of routing and the gated activation against differences, and of the
formats against their definitions (CPU)."""
import numpy as np
import pytest

import experts_ref as ref


@pytest.mark.parametrize("softmax", (True, False))
@pytest.mark.parametrize("renorm", (True, False))
def test_route_gradient_against_differences(softmax, renorm):
    rng = np.random.default_rng(5)
    x = rng.normal(size=(4, 12))
    topk, _ = ref.choose(x, 3, softmax, None, 1, 1, 1, ref.LOWEST["f32"])
    dg = rng.normal(size=(4, 3))
    f = lambda z: (dg * ref.gates(z, topk, softmax, renorm, 2.5, ref.LOWEST["f32"])).sum()  # noqa: E731
    got = ref.route_bwd(x, topk, dg, softmax, renorm, 2.5, ref.LOWEST["f32"])
    eps = 1e-5
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        # central differences: error eps^2/6 f''' + 1e-16 f / eps, both below 1e-9
        assert abs((f(a) - f(b)) / (2 * eps) - got[i]) < 1e-9


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(6)
    h, da = rng.normal(size=(3, 10)), rng.normal(size=(3, 5))
    got = ref.swiglu_bwd(h, da)
    eps = 1e-5
    for i in np.ndindex(h.shape):
        a, b = h.copy(), h.copy()
        a[i] += eps
        b[i] -= eps
        assert abs(((ref.swiglu(a) - ref.swiglu(b)) * da).sum() / (2 * eps) - got[i]) < 1e-9


def test_formats_hold_the_largest_magnitude_and_round_to_nearest():
    rng = np.random.default_rng(7)
    x = rng.normal(size=(40, 64)) * np.exp2(rng.integers(-30, 30, size=(40, 1)))
    x[0] = 0
    x[1, 5] = np.inf
    for enc, val, top, grid in ((ref.mx4, ref.mx4_values, 6.0, ref.E2M1),
                                (ref.mx8, ref.mx8_values, 127.0, np.arange(128.0))):
        c, b = enc(x)
        v = val(c, b).reshape(40, 2, 32)
        w = x.reshape(40, 2, 32)
        assert np.isnan(v[1, 0]).all() and b[1, 0] == 255
        for t, j in np.ndindex(40, 2):
            if (t, j) == (1, 0):
                continue
            s = np.ldexp(1.0, int(b[t, j]) - 127)
            amax = np.abs(w[t, j]).max()
            assert amax <= top * s and (b[t, j] == 0 or amax > top * s / 2)
            near = np.abs(np.abs(w[t, j])[:, None] / s - grid).min(1)
            assert np.allclose(np.abs(v[t, j] - w[t, j]) / s, near, rtol=0, atol=1e-12)
