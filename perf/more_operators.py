"""Benchmark cases of the operators between a layer's projections and behind its adapter
gradients: norms of queries and keys per head with the rotary position embedding (forward
and backward), attention over packed sequences (forward, and the backward that recomputes
the probabilities), and the gradient norm over many tensors with clipping.

``own`` false: ``run`` computes an operator by elementary FP32 torch operations.
``own`` true: ``run`` calls the library as a training step does, writing into buffers
that the program keeps.

Queries are BF16 [T, hq, D], keys and values [T, hk, D] with hq a multiple of hk; query
head h reads key head h // (hq / hk).  The T rows are packed sequences: rows cu[b] to
cu[b + 1] are sequence b.  A sequence may have more keys than queries (a prefix whose keys
are held already); its last query then stands at its last key.
"""
import math

import torch

own = False

EPS = 1e-5
THETA = 500000.0


def listed():
    return [
        # one token of a 32-head model, as in a short continuation
        {"name": "rope 1x32+8x64", "op": "rope", "t": 1, "hq": 32, "hk": 8, "d": 64, "rot": 64,
         "norm": False, "pairs": False, "far": 100000},
        # a training batch of 8 sequences of 1024 tokens, heads of 128 with their norms
        {"name": "rope norm 8192x32+8x128", "op": "rope", "t": 8192, "hq": 32, "hk": 8, "d": 128,
         "rot": 128, "norm": True, "pairs": False, "far": 1024},
        # a packed batch of odd length: neighbouring pairs, half of a head rotated
        {"name": "rope norm bwd 777x8+8x96", "op": "rope_bwd", "t": 777, "hq": 8, "hk": 8, "d": 96,
         "rot": 48, "norm": True, "pairs": True, "far": 4096},
        # the backward pass of 26 sequences of 1024 tokens, 32 and 8 heads of 64
        {"name": "rope norm bwd 26624x32+8x64", "op": "rope_bwd", "t": 26624, "hq": 32, "hk": 8,
         "d": 64, "rot": 64, "norm": True, "pairs": False, "far": 1024},
        # one short prompt
        {"name": "attention 37 4/2x64", "op": "attn", "lens": "37", "prefix": "0", "hq": 4, "hk": 2,
         "d": 64, "causal": True},
        # a packed batch of odd lengths
        {"name": "attention ragged 16/4x96", "op": "attn", "lens": "1,517,129,1900,33,1000",
         "prefix": "0", "hq": 16, "hk": 4, "d": 96, "causal": True},
        # a training batch of 26 sequences of 1024 tokens, 32 and 8 heads of 64
        {"name": "attention 26x1024 32/8x64", "op": "attn", "lens": "26*1024", "prefix": "0",
         "hq": 32, "hk": 8, "d": 64, "causal": True},
        # one long document
        {"name": "attention 16384 16/4x128", "op": "attn", "lens": "16384", "prefix": "0", "hq": 16,
         "hk": 4, "d": 128, "causal": True},
        # the backward pass of a packed batch that sees both directions
        {"name": "attention bwd ragged 8/8x128", "op": "attn_bwd", "lens": "1,517,129,1100,33,700",
         "prefix": "0", "hq": 8, "hk": 8, "d": 128, "causal": False},
        # the backward pass of a training batch of 8 sequences of 1024 tokens
        {"name": "attention bwd 8x1024 32/8x128", "op": "attn_bwd", "lens": "8*1024", "prefix": "0",
         "hq": 32, "hk": 8, "d": 128, "causal": True},
        # the adapters of one layer, rank 16
        {"name": "clip 1 layer", "op": "clip", "layers": 1, "hidden": 2048, "kv": 512,
         "inter": 8192, "r": 16, "over": 4.0},
        # the adapters of 32 layers, rank 32
        {"name": "clip 32 layers", "op": "clip", "layers": 32, "hidden": 4096, "kv": 1024,
         "inter": 14336, "r": 32, "over": 4.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_ROPE = 26624 * 40 * 64
MOST_PAIRS = 16384 * 16384 * 16 * 128          # queries x keys x heads x width, forward
MOST_PAIRS_BWD = 8 * 1024 * 1024 * 32 * 128
MOST_VALUES = 26624 * 32 * 64


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "attn", "attn", "attn_bwd", "attn_bwd", "clip"])
    if op == "clip":
        hidden = _log(rng, 256, 4096) // 16 * 16
        return {"op": op, "layers": _log(rng, 1, 32), "hidden": hidden, "kv": hidden // 4,
                "inter": hidden * 7 // 2, "r": rng.choice([4, 8, 12, 16, 32]),
                "over": rng.choice([0.5, 4.0, 30.0])}
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([64, 64, 80, 96, 112, 128, 128])
    if op in ("rope", "rope_bwd"):
        t = max(1, min(_log(rng, 1, 32768), MOST_ROPE // ((hq + hk) * d)))
        return {"op": op, "t": t, "hq": hq, "hk": hk, "d": d, "rot": rng.choice([d, d, d // 32 * 16]),
                "norm": rng.random() < 0.7, "pairs": rng.random() < 0.4,
                "far": rng.choice([512, 8192, 1000000])}
    most = MOST_PAIRS if op == "attn" else MOST_PAIRS_BWD
    b = _log(rng, 1, 24)
    longest = _log(rng, 1, 8192)
    prefix = rng.choice([0, 0, 0, _log(rng, 1, 2048)])
    while b > 1 and (b * longest * (longest + prefix) * hq * d > most
                     or b * (longest + prefix) * hq * d > MOST_VALUES):
        b -= 1
    while longest * (longest + prefix) * hq * d > most or (longest + prefix) * hq * d > MOST_VALUES:
        longest = longest * 3 // 4
    lens = [longest] + [rng.randint(1, longest) for _ in range(b - 1)]
    rng.shuffle(lens)
    return {"op": op, "lens": ",".join(map(str, lens)), "prefix": str(prefix), "hq": hq, "hk": hk,
            "d": d, "causal": rng.random() < 0.75}


def _lens(case):
    """Query and key lengths of the sequences."""
    lens = []
    for part in case["lens"].split(","):
        n, _, length = part.rpartition("*")
        lens += [int(length)] * int(n or 1)
    return lens, [n + int(case["prefix"]) for n in lens]


def _shapes(case):
    """The adapters' shapes, A [in, r] and B [r, out] of the seven projections of a layer."""
    h, kv, i, r = case["hidden"], case["kv"], case["inter"], case["r"]
    layer = []
    for d_in, d_out in ((h, h), (h, kv), (h, kv), (h, h), (h, i), (h, i), (i, h)):
        layer += [(d_in, r), (r, d_out)]
    return layer * case["layers"]


def work(case):
    op = case["op"]
    if op in ("rope", "rope_bwd"):
        n = case["t"] * (case["hq"] + case["hk"]) * case["d"]
        back = op == "rope_bwd" and case["norm"]
        return {"bytes": (6 if back else 4) * n + 4 * case["t"], "flops": (20 if case["norm"] else 6) * n}
    if op == "clip":
        n = sum(a * b for a, b in _shapes(case))
        return {"bytes": 8 * n, "flops": 3 * n}
    lq, lk = _lens(case)
    if case["causal"]:
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(lq, lk))
    else:
        pairs = sum(q * k for q, k in zip(lq, lk))
    tq, tk, hq, hk, d = sum(lq), sum(lk), case["hq"], case["hk"], case["d"]
    if op == "attn":
        return {"bytes": 2 * d * (2 * tq * hq + 2 * tk * hk) + 4 * tq * hq,
                "flops": 4.0 * d * hq * pairs}
    return {"bytes": 2 * d * (4 * tq * hq + 4 * tk * hk) + 4 * tq * hq, "flops": 10.0 * d * hq * pairs}


# ---------------------------------------------------------------- inputs
def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=g.device, dtype=torch.float32) * std


def _cu(lens, dev):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(dev)


def _inv_freq(rot):
    """Radians per position of each rotated pair."""
    return THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = _gen(seed, dev)
    op = case["op"]
    s = {"op": op}
    if op == "clip":
        shapes = _shapes(case)
        n = sum(a * b for a, b in shapes)
        # the gradients lie in one buffer, as an optimizer keeps them
        s["flat"] = _normal(g, (n,), 1e-3)
        s["max_norm"] = 1e-3 * math.sqrt(n) / case["over"]
        s["out"] = torch.empty_like(s["flat"])
        s["norm"] = torch.empty(1, dtype=torch.float32, device=dev)
        s["ends"] = []
        at = 0
        for a, b in shapes:
            s["ends"].append((at, a, b))
            at += a * b
        s["plan"] = None
        return s
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if op in ("rope", "rope_bwd"):
        t = case["t"]
        s.update(rot=case["rot"], pairs=case["pairs"], norm=case["norm"], inv_freq=_inv_freq(case["rot"]).to(dev))
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=dev, dtype=torch.int32)
        s["q"], s["k"] = _normal(g, (t, hq, d)).bfloat16(), _normal(g, (t, hk, d), 2.0).bfloat16()
        s["gq"] = (1.0 + _normal(g, (d,), 0.1)).bfloat16() if case["norm"] else None
        s["gk"] = (1.0 + _normal(g, (d,), 0.1)).bfloat16() if case["norm"] else None
        if op == "rope_bwd":
            s["dyq"], s["dyk"] = (_normal(g, (t, h, d), 1e-2).bfloat16() for h in (hq, hk))
            s["dgq"], s["dgk"] = (torch.empty(d, dtype=torch.float32, device=dev) for _ in range(2))
        s["oq"], s["ok"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["turns"] = None
        return s
    lq, lk = _lens(case)
    s.update(causal=case["causal"], lq=max(lq), lk=max(lk), cu_q=_cu(lq, dev), cu_k=_cu(lk, dev),
             scale=d ** -0.5)
    tq, tk = sum(lq), sum(lk)
    s["q"], s["k"], s["v"] = (_normal(g, (t, h, d)).bfloat16()
                              for t, h in ((tq, hq), (tk, hk), (tk, hk)))
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((hq, tq), dtype=torch.float32, device=dev)
    if op == "attn_bwd":
        s["do"] = _normal(g, (tq, hq, d), 1e-2).bfloat16()
        s["o"], s["lse"] = _attention(s)  # what the forward pass has left
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[n]) for n in ("q", "k", "v"))
    return s


# ---------------------------------------------------------------- the plain forms
def _turned(x, s, back=False):
    """x [t, heads, d] with its first rot columns turned by the positions' angles."""
    rot, h = s["rot"], s["rot"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"]  # FP32 loses far positions
    c, si = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if back:
        si = -si
    if s["pairs"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        head = torch.stack((a * c - b * si, b * c + a * si), -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:rot]
        head = torch.cat((a * c - b * si, b * c + a * si), -1)
    return torch.cat((head, x[..., rot:]), -1)


def _rope(x, gamma, s):
    x = x.float()
    if gamma is not None:
        x = x * (1.0 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()) * gamma.float()
    return _turned(x, s).bfloat16()


def _rope_bwd(x, gamma, dy, s):
    g = _turned(dy.float(), s, back=True)
    if gamma is None:
        return g.bfloat16(), None
    x = x.float()
    rstd = 1.0 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    n = x * rstd
    dn = g * gamma.float()
    return (rstd * (dn - n * (dn * n).mean(-1, keepdim=True))).bfloat16(), (g * n).double().sum((0, 1)).float()


def _spread(x, cu, most):
    """Packed rows [t, heads, d] as FP32 [b, heads, most, d], zeros behind each sequence."""
    at = cu[:-1, None] + torch.arange(most, device=x.device)
    inside = at < cu[1:, None]
    y = x[at.clamp(max=x.shape[0] - 1)].float() * inside[:, :, None, None]
    return y.transpose(1, 2), inside


def _visible(s, in_q, in_k):
    """[b, 1, lq, lk]: whether a query sees a key."""
    see = in_q[:, :, None] & in_k[:, None, :]
    if s["causal"]:
        ahead = (s["cu_k"].diff() - s["cu_q"].diff())[:, None, None]
        i = torch.arange(s["lq"], device=see.device)[None, :, None]
        j = torch.arange(s["lk"], device=see.device)[None, None, :]
        see = see & (j <= i + ahead)
    return see[:, None]


def _scores(s):
    q, in_q = _spread(s["q"], s["cu_q"], s["lq"])
    k, in_k = _spread(s["k"], s["cu_k"], s["lk"])
    v, _ = _spread(s["v"], s["cu_k"], s["lk"])
    b, hq, lq, d = q.shape
    hk = k.shape[1]
    sc = (q.reshape(b, hk, -1, d) @ k.transpose(2, 3)).view(b, hq, lq, -1).mul_(s["scale"])
    see = _visible(s, in_q, in_k)
    return q, k, v, in_q, sc.masked_fill_(~see, -math.inf)


def _packed(x, inside, like):
    """The inverse of _spread, rounded to BF16."""
    return x.transpose(1, 2)[inside].to(like.dtype)


def _attention(s):
    _, _, v, in_q, sc = _scores(s)
    b, hq, lq, lk = sc.shape
    top = sc.amax(-1, keepdim=True).clamp_min(-3e38)  # a row that sees nothing
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, v.shape[1], -1, lk) @ v).view(b, hq, lq, -1) / total.clamp_min(1e-37)
    lse = (top + total.log())[..., 0]
    return _packed(o, in_q, s["q"]), lse.transpose(1, 2)[in_q].t().contiguous()


def _attention_bwd(s):
    q, k, v, in_q, sc = _scores(s)
    b, hq, lq, lk = sc.shape
    hk = k.shape[1]
    do, _ = _spread(s["do"], s["cu_q"], s["lq"])
    o, _ = _spread(s["o"], s["cu_q"], s["lq"])
    delta = (do * o).sum(-1, keepdim=True)
    lse = sc.new_full((b, lq, hq), math.inf)
    lse[in_q] = s["lse"].t()
    p = sc.sub_(lse.transpose(1, 2)[..., None]).exp_()
    _, in_k = _spread(s["k"], s["cu_k"], s["lk"])
    dv = p.view(b, hk, -1, lk).transpose(2, 3) @ do.reshape(b, hk, -1, do.shape[-1])
    dp = (do.reshape(b, hk, -1, do.shape[-1]) @ v.transpose(2, 3)).view(b, hq, lq, lk)
    ds = dp.sub_(delta).mul_(p).mul_(s["scale"]).view(b, hk, -1, lk)
    dq = (ds @ k).view(b, hq, lq, -1)
    dk = ds.transpose(2, 3) @ q.reshape(b, hk, -1, q.shape[-1])
    return _packed(dq, in_q, s["q"]), _packed(dk, in_k, s["k"]), _packed(dv, in_k, s["v"])


def _plain(s):
    if s["op"] == "rope":
        return _rope(s["q"], s["gq"], s), _rope(s["k"], s["gk"], s)
    if s["op"] == "rope_bwd":
        dq, dgq = _rope_bwd(s["q"], s["gq"], s["dyq"], s)
        dk, dgk = _rope_bwd(s["k"], s["gk"], s["dyk"], s)
        return dq, dk, dgq, dgk
    if s["op"] == "attn":
        return _attention(s)
    if s["op"] == "attn_bwd":
        return _attention_bwd(s)
    norm = s["flat"].double().square().sum().sqrt().float()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return norm.reshape(1), s["flat"] * coef


# ---------------------------------------------------------------- the library's calls
def _library(s):
    import nvfp4_frozen_projection_gb300 as pk
    if s["op"] in ("rope", "rope_bwd"):
        if s["turns"] is None:  # made once, like a model's buffers
            s["turns"] = pk.pact_rope_turns(s["inv_freq"])
        if s["op"] == "rope":
            return pk.pact_qk_norm_rope(s["q"], s["k"], s["positions"], s["turns"], gamma_q=s["gq"],
                                        gamma_k=s["gk"], eps=EPS, interleaved=s["pairs"],
                                        q_out=s["oq"], k_out=s["ok"])
        own_x = s["norm"]
        return pk.pact_qk_norm_rope_bwd(
            s["dyq"], s["dyk"], s["positions"], s["turns"], q=s["q"] if own_x else None,
            k=s["k"] if own_x else None, gamma_q=s["gq"], gamma_k=s["gk"], eps=EPS,
            interleaved=s["pairs"], dq=s["oq"], dk=s["ok"], dgamma_q=s["dgq"] if own_x else None,
            dgamma_k=s["dgk"] if own_x else None)
    if s["op"] == "attn":
        return pk.pact_attention_fwd(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"],
                                     causal=s["causal"], scale=s["scale"], o=s["o"], lse=s["lse"])
    if s["op"] == "attn_bwd":
        return pk.pact_attention_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu_q"],
                                     s["cu_k"], causal=s["causal"], scale=s["scale"], dq=s["dq"],
                                     dk=s["dk"], dv=s["dv"])
    if s["plan"] is None:  # the lists of gradients that an optimizer keeps
        s["plan"] = tuple(pk.GradList([t[at:at + a * b].view(a, b) for at, a, b in s["ends"]])
                          for t in (s["flat"], s["out"]))
    grads, out = s["plan"]
    return pk.pact_clip_grad_norm(grads, s["max_norm"], norm=s["norm"], out=out), s["out"]


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_turn(x, s, sign):
    rot = s["rot"]
    z = s["positions"].double()[:, None] * s["inv_freq"]
    z = torch.polar(torch.ones_like(z), sign * z)[:, None]
    y = x.clone()
    if s["pairs"]:
        w = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * z
        y[..., 0:rot:2], y[..., 1:rot:2] = w.real, w.imag
    else:
        w = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
        y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
    return y


def _exact_rope(x, gamma, dy, s):
    x = x.double()
    if dy is None:
        if gamma is not None:
            x = torch.einsum("thd,th,d->thd", x, (x.pow(2).sum(-1) / x.shape[-1] + EPS).rsqrt(), gamma.double())
        return _exact_turn(x, s, 1.0), None
    g = _exact_turn(dy.double(), s, -1.0)
    if gamma is None:
        return g, None
    r = (x.pow(2).sum(-1) / x.shape[-1] + EPS).rsqrt()
    dn = g * gamma.double()
    dot = torch.einsum("thd,thd->th", dn, x)
    dx = dn * r[..., None] - x * (dot * r ** 3 / x.shape[-1])[..., None]
    return dx, torch.einsum("thd,thd,th->d", g, x, r)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "clip":
        g = s["flat"].double()
        norm = torch.linalg.vector_norm(g)
        coef = s["max_norm"] / (float(norm) + 1e-6)
        return norm.reshape(1), g * min(1.0, coef)
    if op in ("rope", "rope_bwd"):
        q, dgq = _exact_rope(s["q"], s["gq"], s.get("dyq"), s)
        k, dgk = _exact_rope(s["k"], s["gk"], s.get("dyk"), s)
        return (q, k) if op == "rope" else (q, k, dgq, dgk)
    # sequence by sequence and head by head
    lq, lk = _lens(case)
    group = case["hq"] // case["hk"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=o.device)
    dq = torch.zeros_like(o)
    dk = torch.zeros(s["k"].shape, dtype=torch.float64, device=o.device)
    dv = torch.zeros_like(dk)
    aq = ak = 0
    for nq, nk in zip(lq, lk):
        for h in range(case["hq"]):
            q = s["q"][aq:aq + nq, h].double()
            k, v = (s[n][ak:ak + nk, h // group].double() for n in ("k", "v"))
            z = q @ k.t() * s["scale"]
            if case["causal"]:
                z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(nk - nq + 1), -math.inf)
            p = torch.softmax(z, 1)
            if op == "attn":
                o[aq:aq + nq, h] = p @ v
                lse[h, aq:aq + nq] = torch.logsumexp(z, 1)
                continue
            do = s["do"][aq:aq + nq, h].double()
            dp = do @ v.t()
            dz = p * (dp - (p * dp).sum(1, keepdim=True)) * s["scale"]
            dq[aq:aq + nq, h] = dz @ k
            dk[ak:ak + nk, h // group] += dz.t() @ q
            dv[ak:ak + nk, h // group] += p.t() @ do
        aq, ak = aq + nq, ak + nk
    return (o, lse) if op == "attn" else (dq, dk, dv)
