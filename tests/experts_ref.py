"""Plain 64-bit (numpy) forms of routing, the gated activation with its checkpoint, and the
4-bit microscaled format and product. Test infrastructure; shares no code with the library."""
import numpy as np

LOWEST = {"f32": -float(np.finfo(np.float32).max), "bf16": -3.3895313892515355e38}


# ----------------------------------------------------------------------------- routing
def scores(x, softmax, lowest):
    """Scores [T, E] of fp64 logits; masked experts score 0."""
    masked = ~(x > lowest) | (x == np.inf)
    if softmax:
        top = np.max(np.where(masked, -np.inf, x), axis=1, keepdims=True)
        e = np.where(masked, 0.0, np.exp(np.where(masked, 0.0, x) - np.where(np.isfinite(top), top, 0.0)))
        z = e.sum(1, keepdims=True)
        return np.where(z > 0, e / np.where(z > 0, z, 1.0), 0.0), masked
    with np.errstate(over="ignore"):
        s = np.where(masked, 0.0, 1.0 / (1.0 + np.exp(-np.where(masked, 0.0, x))))
    return s, masked


def choose(x, K, softmax, bias, groups, top_groups, group_top, lowest):
    """topk [T, K], by sorting (key descending, index ascending); also the smallest gap between two
    different keys or group scores that the choice compared."""
    T, E = x.shape
    s, masked = scores(x, softmax, lowest)
    by_score = bias is not None or (groups > 1 and group_top > 1)
    key = np.where(masked, -np.inf, s + (0 if bias is None else bias) if by_score else x)
    out = np.zeros((T, K), np.int64)
    gap = np.inf
    m = E // groups
    for t in range(T):
        k = key[t]
        allowed = np.ones(E, bool)
        if groups > 1:
            gs = []
            for g in range(groups):
                v = np.sort(k[g * m:(g + 1) * m])[::-1][:group_top]
                v = v[np.isfinite(v)]
                gs.append(v.sum() if len(v) else -np.inf)
            gs = np.array(gs)
            order = np.lexsort((np.arange(groups), -gs))
            kept = order[:top_groups]
            if top_groups < groups and np.isfinite(gs[order[top_groups]]):
                d = gs[order[top_groups - 1]] - gs[order[top_groups]]
                gap = min(gap, d) if d > 0 else gap
            allowed = np.isin(np.arange(E) // m, kept)
        rank = np.where(allowed, np.where(np.isfinite(k), 0, 1), 2)
        order = np.lexsort((np.arange(E), -np.where(np.isfinite(k), k, 0.0), rank))
        out[t] = order[:K]
        lead = k[order[:K + 1]]
        d = -np.diff(lead[np.isfinite(lead)])
        if (d > 0).any():
            gap = min(gap, d[d > 0].min())
    return out, gap


def gates(x, topk, softmax, renorm, scale, lowest):
    s, _ = scores(x, softmax, lowest)
    v = np.take_along_axis(s, topk, 1)
    if renorm:
        z = v.sum(1, keepdims=True)
        v = np.where(z > 0, v / np.where(z > 0, z, 1.0), 0.0)
    return scale * v


def route_bwd(x, topk, dg, softmax, renorm, scale, lowest):
    """dL/dx for L = sum dg * gates, through the Jacobians."""
    s, _ = scores(x, softmax, lowest)
    v = np.take_along_axis(s, topk, 1)
    dv = scale * dg
    if renorm:
        z = v.sum(1, keepdims=True)
        zi = np.where(z > 0, 1.0 / np.where(z > 0, z, 1.0), 0.0)
        dv = zi * (dv - (dv * v).sum(1, keepdims=True) * zi)
    ds = np.zeros_like(s)
    np.put_along_axis(ds, topk, dv, 1)
    if softmax:
        return s * (ds - (s * ds).sum(1, keepdims=True))
    return ds * s * (1 - s)


# ----------------------------------------------------------------------------- formats
def _exponents(amax, top):
    e = np.full(amax.shape, -127, np.int64)
    pos = amax > 0
    with np.errstate(divide="ignore"):
        guess = np.ceil(np.log2(np.where(pos, amax, 1.0) / top)).astype(np.int64)
    for d in (1, 0, -1, -2):   # the smallest exponent that holds amax, by comparison
        c = guess + d
        e = np.where(pos & (np.ldexp(top, np.clip(c, -1000, 1000)) >= amax), c, e)
    return np.maximum(e, -127)


def _half_even(v, grid):
    a = np.abs(v)
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")
    idx = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
    return idx


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def mx4(x):
    """fp64 [..., n] -> (codes [..., n] 0..15, scale bytes [..., n/32])."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    e = _exponents(np.abs(b).max(-1), 6.0)
    v = np.ldexp(b, -e[..., None])
    codes = _half_even(v, E2M1) + 8 * np.signbit(b)
    codes = np.where(bad[..., None], 0, codes)
    return codes.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def _pow2(byte):
    return np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))


def mx4_values(codes, byte):
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return (v.reshape(*byte.shape, 32) * _pow2(byte)[..., None]).reshape(codes.shape)


def mx8(x):
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    e = _exponents(np.abs(b).max(-1), 127.0)
    q = np.rint(np.ldexp(b, -e[..., None]))
    return q.reshape(x.shape).astype(np.int8), np.where(bad, 255, e + 127).astype(np.uint8)


def mx8_values(q, byte):
    return (q.astype(np.float64).reshape(*byte.shape, 32) * _pow2(byte)[..., None]).reshape(q.shape)


def unpack4(packed):
    """[..., n/2] bytes -> [..., n] codes, the even element from the low 4 bits."""
    return np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)


def unblock_scales(sc, Hp, nblk):
    """[E, MT, KB, 512] -> [E, H', nblk]."""
    E, MT, KB, _ = sc.shape
    v = sc.reshape(E, MT, KB, 32, 4, 4)              # n % 32, n // 32, block
    v = v.transpose(0, 1, 4, 3, 2, 5).reshape(E, MT * 128, KB * 4)
    return v[:, :Hp, :nblk]


# ----------------------------------------------------------------------------- activation
def _sigmoid(g):
    with np.errstate(over="ignore", invalid="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(h):
    F = h.shape[1] // 2
    with np.errstate(invalid="ignore"):
        return h[:, :F] * _sigmoid(h[:, :F]) * h[:, F:]


def swiglu_bwd(h, da):
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    s = _sigmoid(g)
    with np.errstate(invalid="ignore"):
        return np.concatenate((da * u * s * (1 + g * (1 - s)), da * g * s), 1)
