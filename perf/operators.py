"""Benchmark cases of the FP8 (E4M3, one scale per block of 128) operators: the
quantiser, RMSNorm with the residual's addition (forward and backward) and the matrix
product (forward and input gradient).

``own`` false: ``run`` computes an operator by elementary FP32 torch operations.
``own`` true: ``run`` calls the library as a training step or a decoding loop does,
writing into buffers that the program keeps.

An FP8 activation [M, K] is E4M3 values [M, K] and FP32 scales [ceil(K/128), M]; an FP8
weight [N, K] is E4M3 values and FP32 scales [ceil(N/128), ceil(K/128)].
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
T_MIN = E4M3_MAX * 2.0 ** -126  # the smallest block maximum that a scale is made for
EPS = 1e-5


def listed():
    return [
        # one token's activation, quantised while decoding
        {"name": "quant 1x2048", "op": "quant", "m": 1, "k": 2048, "grad": False},
        # a ragged batch: the last block of a row holds 16 values
        {"name": "quant 777x1040", "op": "quant", "m": 777, "k": 1040, "grad": False},
        # the output gradient of the fused gate|up projection of a training step
        {"name": "quant 8192x16384", "op": "quant", "m": 8192, "k": 16384, "grad": True},
        # one token's hidden state
        {"name": "norm 1x2048", "op": "norm", "m": 1, "h": 2048, "residual": True},
        # the hidden states of a training batch of 26 sequences of 1024 tokens
        {"name": "norm 26624x2048", "op": "norm", "m": 26624, "h": 2048, "residual": True},
        # a packed batch of odd length
        {"name": "norm bwd 1333x1040", "op": "norm_bwd", "m": 1333, "h": 1040, "dres": True},
        # the backward pass of a training batch
        {"name": "norm bwd 8192x4096", "op": "norm_bwd", "m": 8192, "h": 4096, "dres": True},
        # a single token through a down projection
        {"name": "linear 1x2048x8192", "op": "linear", "m": 1, "n": 2048, "k": 8192, "add": True},
        # a decoding batch through the fused gate|up projection
        {"name": "linear 24x16384x2048", "op": "linear", "m": 24, "n": 16384, "k": 2048,
         "add": False},
        # a training batch through the down projection, with the residual
        {"name": "linear 8192x4096x8192", "op": "linear", "m": 8192, "n": 4096, "k": 8192,
         "add": True},
        # the input gradient of a packed batch of odd length and ragged widths
        {"name": "dgrad 333x1040x2064", "op": "dgrad", "m": 333, "n": 1040, "k": 2064,
         "add": False},
        # a training batch's through the gate|up projection, added to another branch's
        {"name": "dgrad 8192x16384x2048", "op": "dgrad", "m": 8192, "n": 16384, "k": 2048,
         "add": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return max(lo, _log(rng, lo, hi) // 16 * 16)


def draw(rng):
    op = rng.choice(["quant", "norm", "norm_bwd", "linear", "linear", "dgrad"])
    if op == "quant":
        k = _width(rng, 64, 16384)
        m = min(_log(rng, 1, 32768), 8192 * 16384 // k)
        return {"op": op, "m": m, "k": k, "grad": rng.random() < 0.5}
    if op in ("norm", "norm_bwd"):
        h = _width(rng, 64, 16384)
        most = 26624 * 2048 if op == "norm" else 8192 * 4096
        m = min(_log(rng, 1, 32768), most // h)
        return {"op": op, "m": m, "h": h, "residual" if op == "norm" else "dres": rng.random() < 0.75}
    n, k = _width(rng, 64, 16384), _width(rng, 64, 16384)
    m = max(1, min(_log(rng, 1, 16384), 8192 * 4096 * 8192 // (n * k)))
    return {"op": op, "m": m, "n": n, "k": k, "add": rng.random() < 0.5}


def work(case):
    m = case["m"]

    def act(c):  # bytes of an FP8 activation [m, c]
        return m * c + 4 * m * -(-c // BLOCK)

    if case["op"] == "quant":
        return {"bytes": 2 * m * case["k"] + act(case["k"]), "flops": 3 * m * case["k"]}
    if case["op"] == "norm":
        h, add = case["h"], case["residual"]
        return {"bytes": 2 * m * h + (4 * m * h if add else 0) + 2 * h + act(h) + 4 * m,
                "flops": 8 * m * h}
    if case["op"] == "norm_bwd":
        h = case["h"]
        return {"bytes": (8 if case["dres"] else 6) * m * h + 6 * h + 4 * m, "flops": 12 * m * h}
    n, k = case["n"], case["k"]
    red, out = (k, n) if case["op"] == "linear" else (n, k)
    weight = n * k + 4 * -(-n // BLOCK) * -(-k // BLOCK)
    return {"bytes": act(red) + weight + (4 if case["add"] else 2) * m * out,
            "flops": 2.0 * m * n * k}


# ---------------------------------------------------------------- inputs
def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=g.device, dtype=torch.float32) * std


def _activation(g, m, k):
    """BF16 activations with a few outlier channels (0.1 % of them, 20 times as large)."""
    x = _normal(g, (m, k))
    x[:, torch.randint(0, k, (max(1, k // 1000),), generator=g, device=g.device)] *= 20.0
    return x.bfloat16()


def _gradient(g, m, k):
    """BF16 gradients; one row in eight (a padded or masked token) is zero."""
    dy = _normal(g, (m, k), 1e-2)
    dy[torch.rand(m, generator=g, device=g.device) < 0.125] = 0.0
    return dy.bfloat16()


def _empty_act(m, c, device):
    return (torch.empty((m, c), dtype=torch.float8_e4m3fn, device=device),
            torch.empty((-(-c // BLOCK), m), dtype=torch.float32, device=device))


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = _gen(seed, dev)
    m = case["m"]
    s = {"op": case["op"]}
    if case["op"] == "quant":
        k = case["k"]
        s["x"] = (_gradient if case["grad"] else _activation)(g, m, k)
        s["q"], s["s"] = _empty_act(m, k, dev)
    elif case["op"] == "norm":
        h = case["h"]
        s["x"] = _activation(g, m, h)
        s["residual"] = _normal(g, (m, h), 3.0).bfloat16() if case["residual"] else None
        s["gamma"] = (1.0 + _normal(g, (h,), 0.1)).bfloat16()
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["q"], s["s"] = _empty_act(m, h, dev)
        s["rstd"] = torch.empty(m, dtype=torch.float32, device=dev)
    elif case["op"] == "norm_bwd":
        h = case["h"]
        s["h"] = _activation(g, m, h)
        s["gamma"] = (1.0 + _normal(g, (h,), 0.1)).bfloat16()
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["dy"] = _gradient(g, m, h)
        s["dres"] = _normal(g, (m, h), 1e-2).bfloat16() if case["dres"] else None
        s["dh"] = torch.empty_like(s["dy"])
        s["dgamma"] = torch.empty(h, dtype=torch.float32, device=dev)
    else:
        n, k = case["n"], case["k"]
        red, out = (k, n) if case["op"] == "linear" else (n, k)
        a = _activation(g, m, red) if case["op"] == "linear" else _gradient(g, m, red)
        s["q"], s["s"] = _quant(a.float())
        s["wq"], s["ws"] = _pack(_normal(g, (out, red), 0.02))
        s["add"] = _normal(g, (m, out)).bfloat16() if case["add"] else None
        s["y"] = torch.empty((m, out), dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------- the plain forms
def _blocks(x):
    """[m, k] as [m, ceil(k/128), 128], the last block filled up with zeros."""
    m, k = x.shape
    nb = -(-k // BLOCK)
    if k != nb * BLOCK:
        x = torch.cat([x, x.new_zeros(m, nb * BLOCK - k)], 1)
    return x.view(m, nb, BLOCK)


def _quant(x):
    """E4M3 values and scales of an FP32 [m, k], one scale per 128 values of a row."""
    m, k = x.shape
    b = _blocks(x)
    t = b.abs().amax(2).clamp_min(T_MIN)
    v = b * (E4M3_MAX / t)[:, :, None]
    q = v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(m, -1)[:, :k].contiguous()
    return q, (t / E4M3_MAX).t().contiguous()


def _pack(w):
    """E4M3 values and scales of an FP32 weight [n, k], one scale per 128 x 128 tile."""
    n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    p = w.new_zeros(nb * BLOCK, kb * BLOCK)
    p[:n, :k] = w
    p = p.view(nb, BLOCK, kb, BLOCK)
    t = p.abs().amax((1, 3)).clamp_min(T_MIN)
    v = p * (E4M3_MAX / t)[:, None, :, None]
    q = v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(nb * BLOCK, kb * BLOCK)
    return q[:n, :k].contiguous(), t / E4M3_MAX


def _dequant_act(q, s, dtype=torch.float32):
    k = q.shape[1]
    return q.to(dtype) * s.to(dtype).t().repeat_interleave(BLOCK, 1)[:, :k]


def _dequant_weight(q, s, dtype=torch.float32):
    n, k = q.shape
    s = s.to(dtype).repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return q.to(dtype) * s


def _plain(s):
    if s["op"] == "quant":
        return _quant(s["x"].float())
    if s["op"] == "norm":
        h = s["x"]
        if s["residual"] is not None:
            h = (h.float() + s["residual"].float()).bfloat16()
        f = h.float()
        rstd = 1.0 / (f.square().mean(1) + EPS).sqrt()
        q, sc = _quant(f * rstd[:, None] * s["gamma"].float())
        return (q, sc, rstd) if s["residual"] is None else (q, sc, rstd, h)
    if s["op"] == "norm_bwd":
        n = s["h"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        dn = dy * s["gamma"].float()
        c = (dn * n).mean(1, keepdim=True)
        dh = s["rstd"][:, None] * (dn - n * c)
        if s["dres"] is not None:
            dh = dh + s["dres"].float()
        return dh.bfloat16(), (dy * n).sum(0)
    y = _dequant_act(s["q"], s["s"]) @ _dequant_weight(s["wq"], s["ws"]).t()
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.bfloat16()


# ---------------------------------------------------------------- the library's calls
def _library(s):
    import nvfp4_frozen_projection_gb300 as pk
    if s["op"] == "quant":
        out = pk.pact_quant_fp8(s["x"], out=pk.FP8(s["q"], s["s"]))
        return out.q, out.s
    if s["op"] == "norm":
        h, yq, rstd = pk.pact_add_rmsnorm_quant_fp8(
            s["x"], s["residual"], s["gamma"], EPS, h=s["h"], out=pk.FP8(s["q"], s["s"]),
            rstd=s["rstd"])
        return (yq.q, yq.s, rstd) if s["residual"] is None else (yq.q, yq.s, rstd, h)
    if s["op"] == "norm_bwd":
        return pk.pact_add_rmsnorm_bwd(s["h"], s["gamma"], s["rstd"], s["dy"], dres=s["dres"],
                                       dh=s["dh"], dgamma=s["dgamma"])
    x, w = pk.FP8(s["q"], s["s"]), pk.FP8Weight(s["wq"], s["ws"])
    if s["op"] == "linear":
        return pk.pact_linear_fp8_fwd(x, w, residual=s["add"], y=s["y"])
    return pk.pact_linear_fp8_dgrad(x, w, dx_prev=s["add"], dx=s["y"])


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits
def _e4m3(v):
    """FP64 values rounded to the nearest E4M3 value, ties to even, at most 448."""
    v = v.clamp(-E4M3_MAX, E4M3_MAX)
    _, e = torch.frexp(v)  # |v| = f 2^e, 0.5 <= f < 1: 2^(e-1) is the leading bit
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp_min(-9))
    return torch.where(v == 0, v, torch.round(v / step) * step)


def _exact_quant(x):
    m, k = x.shape
    nb = -(-k // BLOCK)
    p = torch.nn.functional.pad(x, (0, nb * BLOCK - k))
    t = p.reshape(m, nb, BLOCK).abs().max(-1).values.clamp_min(T_MIN)
    q = _e4m3(x * E4M3_MAX / t.repeat_interleave(BLOCK, 1)[:, :k])
    return q, t.t().contiguous() / E4M3_MAX


def exact(case, seed):
    s = {n: (v.double() if isinstance(v, torch.Tensor) and n not in ("q", "wq") else v)
         for n, v in prepare(case, seed).items()}
    if s["op"] == "quant":
        return _exact_quant(s["x"])
    if s["op"] == "norm":
        h = s["x"]
        if s["residual"] is not None:
            h = (h + s["residual"]).float().bfloat16().double()  # the stored sum is BF16
        rstd = (h.pow(2).sum(1) / h.shape[1] + EPS).rsqrt()
        q, sc = _exact_quant(torch.einsum("mh,m,h->mh", h, rstd, s["gamma"]))
        return (q, sc, rstd) if s["residual"] is None else (q, sc, rstd, h)
    if s["op"] == "norm_bwd":
        h, r, dy = s["h"], s["rstd"], s["dy"]
        dot = torch.einsum("mh,mh,h->m", dy, h, s["gamma"])
        dh = (dy * s["gamma"] - h * (dot * r * r / h.shape[1])[:, None]) * r[:, None]
        if s["dres"] is not None:
            dh = dh + s["dres"]
        return dh, torch.einsum("mh,mh,m->h", dy, h, r)
    # block by block: the products of a block of 128, then its two scales
    m, red = s["q"].shape
    out = s["wq"].shape[0]
    y = torch.zeros(m, out, dtype=torch.float64, device=s["q"].device)
    for b in range(-(-red // BLOCK)):
        at = slice(b * BLOCK, min(red, (b + 1) * BLOCK))
        col = s["ws"][:, b].repeat_interleave(BLOCK)[:out]
        y += (s["q"][:, at].double() @ s["wq"][:, at].double().t()) * s["s"][b][:, None] * col
    return y if s["add"] is None else y + s["add"]
