"""Plain 64-bit forms of the FP8 operators, for the tests only: numpy arrays on the
host, each value from its definition."""
import numpy as np

BLOCK = 128
T_MIN = 448.0 * 2.0 ** -126


def blocks_of(k):
    return -(-k // BLOCK)


def per_block(a, fn):
    """fn over the blocks of 128 of each row: [m, ceil(k/128)]."""
    k = a.shape[1]
    return np.stack([fn(a[:, b * BLOCK:min(k, (b + 1) * BLOCK)]) for b in range(blocks_of(k))], 1)


def spread(s, k):
    """[m, ceil(k/128)] block values to the columns they belong to."""
    return np.repeat(s, BLOCK, axis=1)[:, :k]


def e4m3(v):
    """The nearest E4M3 values, ties to even, saturating at 448; float64 in and out."""
    v = np.clip(np.asarray(v, np.float64), -448.0, 448.0)
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    return np.where(v == 0, v, np.rint(v / step) * step)


def quant_fp32(x):
    """(values, scales [blocks, m]) by the definition's FP32 steps; x float32 [m, k]."""
    x = np.asarray(x, np.float32)
    t = np.maximum(per_block(np.abs(x), lambda b: b.max(1)), np.float32(T_MIN)).astype(np.float32)
    s = (t / np.float32(448)).astype(np.float32)
    r = (np.float32(448) / t).astype(np.float32)
    q = e4m3((x * spread(r, x.shape[1])).astype(np.float32))
    return q, np.ascontiguousarray(s.T)


def pack_fp32(w):
    """(values [n, k], scales [ceil(n/128), ceil(k/128)]) of a float32 weight."""
    n, k = w.shape
    rows = per_block(np.abs(w), lambda b: b.max(1))
    t = np.maximum(per_block(np.ascontiguousarray(rows.T), lambda b: b.max(1)).T,
                   np.float32(T_MIN)).astype(np.float32)
    s = (t / np.float32(448)).astype(np.float32)
    r = (np.float32(448) / t).astype(np.float32)
    full = spread(np.repeat(r, BLOCK, axis=0)[:n], k)
    return e4m3((w.astype(np.float32) * full).astype(np.float32)), s


def dequant(q, s):
    return np.asarray(q, np.float64) * spread(np.asarray(s, np.float64).T, q.shape[1])


def dequant_weight(q, s):
    n, k = q.shape
    return np.asarray(q, np.float64) * spread(np.repeat(np.asarray(s, np.float64), BLOCK, 0)[:n], k)


def norm(h, gamma, eps):
    """(y, rstd) of the RMSNorm of h."""
    h = np.asarray(h, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * np.asarray(gamma, np.float64), rstd


def norm_bwd(h, gamma, rstd, dy, dres):
    """(dh, dgamma, and the magnitudes |rstd dn|, |rstd n|, c, mean |dn n|, sum |dy n|)."""
    h, gamma, rstd, dy = (np.asarray(a, np.float64) for a in (h, gamma, rstd, dy))
    n = h * rstd[:, None]
    dn = dy * gamma
    c = (dn * n).mean(1, keepdims=True)
    dh = rstd[:, None] * (dn - n * c)
    if dres is not None:
        dh = dh + np.asarray(dres, np.float64)
    mags = (np.abs(dn) * rstd[:, None], np.abs(n) * rstd[:, None], np.abs(c),
            np.abs(dn * n).mean(1, keepdims=True), np.abs(dy * n).sum(0))
    return dh, (dy * n).sum(0), mags
