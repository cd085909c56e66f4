"""Plain 64-bit forms of the operators on heads (norm and rotation, attention over packed
sequences) and of gradient clipping, and the bounds that their tests use.

Rounding a value to BF16 moves it by at most U = 2^-8 of itself.  Sums of many independent
roundings are bounded two ways: by the sum of the single bounds, which always holds, and by
Hoeffding's inequality, which a sum of n errors, each within b_i, exceeds T sqrt(sum b_i^2)
with a probability of at most 2 exp(-T^2 / 2); T = 7 makes that 5e-11.
"""
import torch

U = 2.0 ** -8      # half a step of BF16, relative
E = 2.0 ** -24     # half a step of FP32, relative
T = 7.0


def turn(x, positions, inv_freq, interleaved, sign=1.0):
    """x [t, heads, D] in 64 bits, its first 2 len(inv_freq) columns turned."""
    rot = 2 * inv_freq.numel()
    z = positions.double()[:, None, None] * inv_freq.double()
    c, s = torch.cos(z), torch.sin(z) * sign
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2),
                                                                     slice(rot // 2, rot))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def spread(x, rot, interleaved):
    """|a| + |b| of each column's pair, |x| behind the turned columns."""
    y = x.abs().clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2),
                                                                     slice(rot // 2, rot))
    y[..., a] = y[..., b] = x[..., a].abs() + x[..., b].abs()
    return y


def rope(x, positions, inv_freq, interleaved, gamma=None, eps=0.0):
    """(y, what an error of relative size 1 before the rotation could move it by)"""
    x = x.double()
    if gamma is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * gamma.double()
    return turn(x, positions, inv_freq, interleaved), spread(x, 2 * inv_freq.numel(), interleaved)


def rope_bwd(dy, positions, inv_freq, interleaved, x=None, gamma=None, eps=0.0):
    """(dx, dgamma, magnitude of dx's terms, sum of |dgamma's terms|)"""
    dy = dy.double()
    g = turn(dy, positions, inv_freq, interleaved, -1.0)
    gs = spread(dy, 2 * inv_freq.numel(), interleaved)
    if gamma is None:
        return g, None, gs, None
    x = x.double()
    rstd = 1.0 / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    n, gm = x * rstd, gamma.double()
    dn = g * gm
    dx = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    mag = rstd * (gs * gm.abs() + n.abs() * (gs * gm.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, (g * n).sum((0, 1)), mag, (gs * n.abs()).sum((0, 1))


def sequences(cu_q, cu_k):
    return list(zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]))


def visible(lq, lk, causal, device):
    see = torch.ones(lq, lk, dtype=torch.bool, device=device)
    return see.tril(lk - lq) if causal else see


def scores(q, k, scale, see):
    s = (q @ k.t()) * scale
    return s.masked_fill(~see, -float("inf"))


def attention(q, k, v, cu_q, cu_k, causal, scale):
    """(o, lse, bound of o's error, bound of lse's), NaN in rows of no sequence.  The bounds
    count the rounding of the probabilities and of the result, and FP32 sums."""
    dev, (tq, hq, d), hk = q.device, q.shape, k.shape[1]
    o = torch.full((tq, hq, d), float("nan"), dtype=torch.float64, device=dev)
    lse = torch.full((hq, tq), float("nan"), dtype=torch.float64, device=dev)
    bo, bl = o.clone(), lse.clone()
    for q0, q1, k0, k1 in sequences(cu_q, cu_k):
        if q1 <= q0:
            continue
        see = visible(q1 - q0, k1 - k0, causal, dev)
        empty = ~see.any(1)
        for h in range(hq):
            x, y, z = (a.double() for a in (q[q0:q1, h], k[k0:k1, h // (hq // hk)],
                                            v[k0:k1, h // (hq // hk)]))
            s = scores(x, y, scale, see)
            if k1 > k0:
                l = torch.logsumexp(s, 1)
                top = s.amax(1)
            else:
                l = top = torch.full((q1 - q0,), -float("inf"), dtype=torch.float64, device=dev)
            p = torch.exp(s - torch.where(empty, 0.0, l)[:, None])
            r = p @ z
            o[q0:q1, h], lse[h, q0:q1] = r, l
            # a score's own error: the product's FP32 sums over D in steps of 16, the exponent's
            # arithmetic, and the exponential's
            a = (x.abs() @ y.abs().t()).amax(1) * scale if k1 > k0 else torch.zeros_like(l)
            ds = E * (2 * (d // 16) * a + 8 * torch.where(empty, 0.0, top).abs() + 16)
            mass = p @ z.abs()
            sq = (p.pow(2) @ z.pow(2)).sqrt()
            many = torch.minimum(mass, T * sq)
            bo[q0:q1, h] = U * (1 + U) * (r.abs() + many) + (2 * ds + 64 * E)[:, None] * mass
            bl[h, q0:q1] = ds + 4 * E * torch.where(empty, 0.0, l).abs()
    return o, lse, bo, bl


def attention_bwd(do, q, k, v, o, lse, cu_q, cu_k, causal, scale):
    """(dq, dk, dv) by the formulas from the given o and lse, and the bounds of their
    errors; NaN in rows of no sequence."""
    dev, (tq, hq, d), (tk, hk, _) = q.device, q.shape, k.shape
    g = hq // hk
    f = dict(dtype=torch.float64, device=dev)
    out = [torch.full(t.shape, float("nan"), **f) for t in (q, k, v)]
    dq, dk, dv = out
    # squares and sums of magnitudes of what is rounded, and of what FP32 sums err by
    many = [torch.zeros(t.shape, **f) for t in (q, k, v)]
    worst = [torch.zeros(t.shape, **f) for t in (q, k, v)]
    fp32 = [torch.zeros(t.shape, **f) for t in (q, k, v)]
    for q0, q1, k0, k1 in sequences(cu_q, cu_k):
        dq[q0:q1] = 0
        dk[k0:k1] = 0
        dv[k0:k1] = 0
        if q1 <= q0 or k1 <= k0:
            continue
        see = visible(q1 - q0, k1 - k0, causal, dev)
        for h in range(hq):
            x, w, r = (a[q0:q1, h].double() for a in (q, do, o))
            y, z = (a[k0:k1, h // g].double() for a in (k, v))
            s = scores(x, y, scale, see)
            l = lse[h, q0:q1].double()
            p = torch.exp(s - torch.where(torch.isinf(l), 0.0, l)[:, None])
            delta = (w * r).sum(1, keepdim=True)
            dp = w @ z.t()
            ds = p * (dp - delta)
            dq[q0:q1, h] = scale * (ds @ y)
            dk[k0:k1, h // g] += scale * (ds.t() @ x)
            dv[k0:k1, h // g] += p.t() @ w
            a = (x.abs() @ y.abs().t()) * scale
            ep = E * (2 * (d // 16) * a + 8 * l.abs().clamp(max=1e30)[:, None] + 16)
            es = p * (ep * (dp - delta).abs() + E * (2 * (d // 16) + 8) *
                      (w.abs() @ z.abs().t() + (w * r).abs().sum(1, keepdim=True)))
            for t, lhs, rhs, at, f32 in ((0, ds, y, (slice(q0, q1), h), es),
                                         (1, ds.t(), x, (slice(k0, k1), h // g), es.t()),
                                         (2, p.t(), w, (slice(k0, k1), h // g), (p * ep).t())):
                c = scale if t < 2 else 1.0
                many[t][at] += (c * c) * (lhs.pow(2) @ rhs.pow(2))
                worst[t][at] += c * (lhs.abs() @ rhs.abs())
                fp32[t][at] += c * (f32 @ rhs.abs())
    bounds = [U * (1 + U) * (a.abs() + torch.minimum(b, T * m.sqrt())) + e + 64 * E * b
              for a, m, b, e in zip(out, many, worst, fp32)]
    return out, bounds


def check(got, want, bound, what):
    """Every value within its bound; NaN in `want`: not looked at."""
    live = ~torch.isnan(want)
    err = (got.double() - want).abs()[live]
    room = bound[live]
    if not err.numel():
        return 0.0
    same = (got.double() == want)[live]
    bad = ~(same | (err <= room))
    worst = float((err / room.clamp_min(1e-300)).nan_to_num(0.0, posinf=0.0).max())
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {err.numel()} outside, worst {worst:.3f}"
    return worst
