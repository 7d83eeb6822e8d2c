"""Plain numpy forms of 8-bit rows and of grouped products. Test infrastructure; shares no code with the library."""
import numpy as np


def quantise(v):
    """fp64 [..., n] of bf16 or fp32 values -> (int64 codes, fp32 scales [...])."""
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    m = np.abs(v).max(-1)
    codes = np.rint(127.0 * v / np.where(m > 0, m, 1.0)[..., None]).astype(np.int64)
    with np.errstate(under="ignore"):
        scales = (m.astype(np.float32) / np.float32(127.0)).astype(np.float32)
    return codes, np.where(bad, np.float32(np.nan), scales)


def bf16_bits(x):
    """fp32 -> bf16 bit patterns, round to nearest even (finite values)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def product_bits(q, scale, wq, w_scale):
    """bf16 bit patterns of one expert's rows where the integer sums are below 2^24: (sum * w_scale) * scale with
    each fp32 rounding. q [rows, H], wq [N, H]."""
    acc = q.astype(np.float64) @ wq.astype(np.float64).T
    assert np.abs(q).astype(np.float64).dot(np.abs(wq).astype(np.float64).T).max(initial=0.0) < 2 ** 24
    with np.errstate(under="ignore"):
        return bf16_bits((acc.astype(np.float32) * w_scale[None, :]) * scale[:, None])
