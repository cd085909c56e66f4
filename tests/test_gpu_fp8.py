"""GPU parity of the FP8 operators against plain 64-bit forms (fp8_ref.py).

Bounds, from the arithmetic alone (u = 2^-24, half an FP32 step; a BF16 store is off by
at most 2^-8 of the value):
  quantiser   the FP32 steps of the definition, bit for bit.
  rstd        a row's sum of squares is added in chains of at most 32 fused steps in a
              lane, 5 over the warp, 15 over the warps; all terms positive: 60 u on the
              sum with the division, 30 u on its root, 3 u for the last operations:
              40 u.  The FP8 output, given that rstd, bit for bit.
  dh          2^-8 of the value, and u times: 4 |rstd dn| (products and sum),
              8 |rstd n c|, and 64 |rstd n| mean |dn n| for the sum c, chains as above.
  dgamma      u (rows / 304 + 80) sum |dy n|: the rows of one of 304 groups in a chain,
              then up to 2432 partial sums, 64 lanes of 38 and 16 joins; or, up to 4096
              rows, 128 lanes of 32 and 11 joins.
  product     2^-8 of the value, and 2^-23 (128 + blocks + 8) sum |x w|: FP32 additions
              of a block in any order, truncated or rounded, then one fused step for
              each block, the scales' product, and the join.
"""
import numpy as np
import pytest
import torch

import fp8_ref as ref
import nvfp4_frozen_projection_gb300 as pk
from nvfp4_frozen_projection_gb300 import FP8, FP8Weight
from nvfp4_frozen_projection_gb300.stack import Fp8Linear

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GUARD = 4096


def bf16(rng, shape, std=1.0):
    a = torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32))
    return a.to(torch.bfloat16).cuda()


def host(t):
    return t.detach().to(torch.float64).cpu().numpy()


def activation(rng, m, k, std=1.0):
    x = bf16(rng, (m, k), std)
    x[:, int(rng.integers(0, k))] *= 20
    return x


class Guarded:
    """A buffer between two guards of a fixed pattern, filled with garbage."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        self.n, self.raw = n, torch.full((n + 2 * GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
        self.raw[GUARD:GUARD + n] = 0x77
        self.t = self.raw[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        r = self.raw.cpu()
        assert bool((r[:GUARD] == 0x5A).all()) and bool((r[GUARD + self.n:] == 0x5A).all())


def guarded_fp8(m, k):
    q, s = Guarded((m, k), torch.float8_e4m3fn), Guarded(FP8.scale_shape(m, k), torch.float32)
    return FP8(q.t, s.t), (q, s)


def assert_fp8_bits(got, q, s):
    assert np.array_equal(got.s.cpu().numpy().view(np.uint32), s.view(np.uint32))
    g = host(got.q)
    assert np.array_equal(g, q) and np.array_equal(np.signbit(g), np.signbit(q))


def random_fp8(rng, m, k, std=1.0):
    return pk.pact_quant_fp8(activation(rng, m, k, std))


def random_weight(rng, n, k, std=0.02):
    w = torch.from_numpy((rng.standard_normal((n, k)) * std).astype(np.float32)).cuda()
    return pk.pact_pack_weight_fp8_fwd(w)


def check_product(y, x, w, add=None):
    a, b = ref.dequant(host(x.q), host(x.s)), ref.dequant_weight(host(w.q), host(w.s))
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if add is not None:
        want, mag = want + host(add), mag + np.abs(host(add))
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -23 * (128 + ref.blocks_of(x.cols) + 8) * mag
    err = np.abs(host(y) - want)
    assert np.all(err <= tol * (1 + 2.0 ** -8)), float((err - tol).max())


# ---------------------------------------------------------------- quantiser and packs
SHAPES = [(1, 16), (1, 2048), (2, 128), (7, 144), (8, 112), (9, 1040), (33, 4096), (64, 16384),
          (257, 2064), (1000, 640)]


@pytest.mark.parametrize("m,k", SHAPES)
def test_quant(m, k):
    rng = np.random.default_rng(m * 7 + k)
    x = activation(rng, m, k)
    if m > 2:
        x[1] = 0.0
        x[2] = -0.0
    out, guards = guarded_fp8(m, k)
    pk.pact_quant_fp8(x, out=out)
    pk.pact_check_status()
    assert_fp8_bits(out, *ref.quant_fp32(x.float().cpu().numpy()))
    for g in guards:
        g.check()


@pytest.mark.parametrize("scale", [2.0 ** -133, 2.0 ** -126, 2.0 ** -100, 2.0 ** 90, 2.0 ** 127])
def test_quant_extreme_magnitudes(scale):
    """From the smallest BF16 subnormal to the largest finite values."""
    rng = np.random.default_rng(5)
    x = (torch.from_numpy(rng.uniform(-1, 1, (16, 384))).double() * scale).float().bfloat16().cuda()
    x[3, :128] = 0.0
    x[3, 17] = torch.finfo(torch.bfloat16).max if scale > 1 else 2.0 ** -133
    out = pk.pact_quant_fp8(x)
    assert_fp8_bits(out, *ref.quant_fp32(x.float().cpu().numpy()))


@pytest.mark.parametrize("ld,off", [(1048, 0), (1040, 8), (2080, 16)])
def test_quant_strided_rows(ld, off):
    """Rows of a wider tensor, starting at a 16-byte boundary inside it."""
    rng = np.random.default_rng(ld)
    m, k = 37, 1024
    big = bf16(rng, (m, ld))
    x = big[:, off:off + k]
    assert_fp8_bits(pk.pact_quant_fp8(x), *ref.quant_fp32(x.float().cpu().numpy()))


def test_quant_offsets_past_32_bits():
    """More than 2^32 values: the last rows are those of a small call on them."""
    m, k = 262208, 16384
    x = torch.empty((m, k), dtype=torch.bfloat16, device="cuda")
    x.view(torch.int16).copy_((torch.arange(k, device="cuda") % 997 + 16000).short())
    x[-3:] = bf16(np.random.default_rng(1), (3, k))
    out = pk.pact_quant_fp8(x)
    tail = pk.pact_quant_fp8(x[-3:].clone())
    assert torch.equal(out.q[-3:].view(torch.uint8), tail.q.view(torch.uint8))
    assert torch.equal(out.s[:, -3:], tail.s)
    first = pk.pact_quant_fp8(x[:3].clone())
    assert torch.equal(out.q[m // 2].view(torch.uint8), first.q[0].view(torch.uint8))


@pytest.mark.parametrize("n,k", [(16, 16), (128, 128), (144, 272), (1040, 2064), (256, 64)])
def test_pack_weight(n, k):
    rng = np.random.default_rng(n + k)
    w = (rng.standard_normal((n, k)) * 0.02).astype(np.float32)
    w[: min(n, 128), : min(k, 128)] *= 0 if n > 128 else 1  # a zero tile
    q, s = ref.pack_fp32(w)
    gq, gs = Guarded((n, k), torch.float8_e4m3fn), Guarded(s.shape, torch.float32)
    f = pk.pact_pack_weight_fp8_fwd(torch.from_numpy(w).cuda(), out=FP8Weight(gq.t, gs.t))
    assert_fp8_bits(f, q, s)
    gq.check(), gs.check()
    gq, gs = Guarded((k, n), torch.float8_e4m3fn), Guarded(s.T.shape, torch.float32)
    b = pk.pact_pack_weight_fp8_bwd(torch.from_numpy(w).cuda(), out=FP8Weight(gq.t, gs.t))
    assert_fp8_bits(b, q.T, np.ascontiguousarray(s.T))
    gq.check(), gs.check()


# ---------------------------------------------------------------- RMSNorm
NORM_SHAPES = [(1, 16), (1, 2048), (3, 128), (5, 144), (9, 256), (130, 1024), (17, 1040),
               (33, 2048), (64, 4096), (31, 5120), (20, 8192), (7, 8208), (5, 12288), (3, 16384),
               (700, 640), (2500, 512)]


@pytest.mark.parametrize("m,h", NORM_SHAPES)
@pytest.mark.parametrize("with_res", [True, False])
def test_add_rmsnorm_quant(m, h, with_res):
    rng = np.random.default_rng(m * 3 + h)
    x, res = activation(rng, m, h), bf16(rng, (m, h), 3.0)
    gamma = (1 + bf16(rng, (h,), 0.1)).bfloat16()
    if m > 2:  # a row of zeros
        x[1] = 0.0
        res[1] = 0.0
    out, guards = guarded_fp8(m, h)
    gh, gr = Guarded((m, h), torch.bfloat16), Guarded((m,), torch.float32)
    eps = 1e-5
    hh, yq, rstd = pk.pact_add_rmsnorm_quant_fp8(x, res if with_res else None, gamma, eps,
                                                 h=gh.t if with_res else None, out=out, rstd=gr.t)
    pk.pact_check_status()
    for g in (*guards, gh, gr):
        g.check()
    want_h = (x.float() + res.float()).bfloat16() if with_res else x
    assert torch.equal(hh, want_h)
    y, want_rstd = ref.norm(host(want_h), host(gamma), np.float64(np.float32(eps)))
    got = host(rstd)
    assert np.all(np.abs(got - want_rstd) <= 40 * U * want_rstd)
    y32 = (want_h.float() * rstd[:, None]) * gamma.float()
    assert_fp8_bits(yq, *ref.quant_fp32(y32.cpu().numpy()))
    # the values themselves: half an E4M3 step of the exact y, and the errors above
    step = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * ref.spread(host(yq.s).T, h))
    assert np.all(np.abs(ref.dequant(host(yq.q), host(yq.s)) - y) <= step * (1 + 2.0 ** -10))


@pytest.mark.parametrize("into", ["x", "residual"])
def test_add_rmsnorm_in_place(into):
    rng = np.random.default_rng(3)
    x, res, gamma = bf16(rng, (70, 2048)), bf16(rng, (70, 2048)), bf16(rng, (2048,))
    h, yq, rstd = pk.pact_add_rmsnorm_quant_fp8(x, res, gamma)
    t = x if into == "x" else res
    h2, yq2, rstd2 = pk.pact_add_rmsnorm_quant_fp8(x, res, gamma, h=t)
    assert h2 is t and torch.equal(h, t) and torch.equal(rstd, rstd2)
    assert torch.equal(yq.q.view(torch.uint8), yq2.q.view(torch.uint8))


@pytest.mark.parametrize("m,h", NORM_SHAPES + [(3000, 1040), (5000, 528), (4097, 64), (1500, 8192),
                                            (700, 10000), (320, 16384), (400, 8208)])
@pytest.mark.parametrize("with_res", [True, False])
def test_add_rmsnorm_bwd(m, h, with_res):
    rng = np.random.default_rng(m * 5 + h)
    hh, dy = activation(rng, m, h), bf16(rng, (m, h), 1e-2)
    gamma = (1 + bf16(rng, (h,), 0.1)).bfloat16()
    dres = bf16(rng, (m, h), 1e-2) if with_res else None
    if m > 2:
        dy[1] = 0.0  # a masked token
        hh[2] = 0.0
    _, _, rstd = pk.pact_add_rmsnorm_quant_fp8(hh, None, gamma)
    gd, gg = Guarded((m, h), torch.bfloat16), Guarded((h,), torch.float32)
    dh, dgamma = pk.pact_add_rmsnorm_bwd(hh, gamma, rstd, dy, dres=dres, dh=gd.t, dgamma=gg.t)
    pk.pact_check_status()
    gd.check(), gg.check()
    want, want_g, (dn, n, c, mean, dyn) = ref.norm_bwd(
        host(hh), host(gamma), host(rstd), host(dy), None if dres is None else host(dres))
    tol = 2.0 ** -8 * np.abs(want) + U * (4 * dn + 8 * n * c + 64 * n * mean
                                          + (0 if dres is None else np.abs(host(dres))))
    assert np.all(np.abs(host(dh) - want) <= tol * (1 + 2.0 ** -8))
    chain = -(-m // 304) + 80
    assert np.all(np.abs(host(dgamma) - want_g) <= U * chain * dyn + 1e-45)
    # without dgamma: the same dh
    again, none = pk.pact_add_rmsnorm_bwd(hh, gamma, rstd, dy, dres=dres)
    assert none is None and torch.equal(again, dh)


@pytest.mark.parametrize("m,h", [(40, 1040), (5000, 528), (30, 8192), (500, 12304)])
def test_add_rmsnorm_bwd_in_place(m, h):
    rng = np.random.default_rng(8)
    hh, dy, dres = (bf16(rng, (m, h)) for _ in range(3))
    gamma = bf16(rng, (h,))
    _, _, rstd = pk.pact_add_rmsnorm_quant_fp8(hh, None, gamma)
    want, dg = pk.pact_add_rmsnorm_bwd(hh, gamma, rstd, dy, dres=dres, dgamma=True)
    for name in ("dy", "dres"):
        d = {"dy": dy.clone(), "dres": dres.clone()}
        got, dg2 = pk.pact_add_rmsnorm_bwd(hh, gamma, rstd, d["dy"], dres=d["dres"], dh=d[name],
                                           dgamma=True)
        assert torch.equal(got, want) and torch.equal(dg, dg2)


def test_add_rmsnorm_gradient_against_differences():
    """<dh, E> and <dgamma, e> against central differences of a 64-bit forward."""
    rng = np.random.default_rng(11)
    m, h, eps = 4, 272, 1e-5
    hh, dy, gamma = bf16(rng, (m, h)), bf16(rng, (m, h)), (1 + bf16(rng, (h,), 0.1)).bfloat16()
    _, _, rstd = pk.pact_add_rmsnorm_quant_fp8(hh, None, gamma, eps)
    dh, dgamma = pk.pact_add_rmsnorm_bwd(hh, gamma, rstd, dy, dgamma=True)
    H, G, D = host(hh), host(gamma), host(dy)

    def loss(a, g):
        return float((ref.norm(a, g, eps)[0] * D).sum())

    t = 1e-5
    for k in range(4):
        E, e = rng.standard_normal((m, h)), rng.standard_normal(h)
        fd = (loss(H + t * E, G) - loss(H - t * E, G)) / (2 * t)
        # each dh is off by at most 2^-8 of itself (and the differences by about t^2)
        assert abs((host(dh) * E).sum() - fd) <= 2.0 ** -8 * np.abs(host(dh) * E).sum() + 1e-4
        fd = (loss(H, G + t * e) - loss(H, G - t * e)) / (2 * t)
        assert abs((host(dgamma) * e).sum() - fd) <= 100 * U * np.abs(host(dgamma) * e).sum() + 1e-4


# ---------------------------------------------------------------- product
PRODUCTS = [(1, 16, 16), (1, 2048, 2048), (2, 1040, 144), (7, 128, 8192), (8, 272, 400),
            (9, 16, 1024), (16, 512, 2064), (17, 2048, 512), (24, 4096, 2048), (32, 1024, 4096),
            (33, 1040, 1040), (64, 2048, 2048), (65, 144, 2064), (127, 1024, 1024),
            (128, 512, 4096), (129, 2064, 656), (200, 1040, 272), (256, 256, 128), (257, 2048, 640),
            (300, 16, 16), (333, 1040, 2064), (512, 4096, 1040), (1000, 1296, 2048),
            (2050, 528, 1168), (2100, 4080, 1040), (2305, 4096, 144),
            # CTAs of a cluster that share a tile: four, three, two; many CTAs of few tokens
            (3, 16384, 2064), (100, 4096, 2192), (120, 4880, 2064), (500, 2048, 4112), (700, 128, 528)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("with_add", [False, True])
def test_linear_fwd(m, n, k, with_add):
    rng = np.random.default_rng(m + 3 * n + 5 * k)
    x, w = random_fp8(rng, m, k), random_weight(rng, n, k)
    add = bf16(rng, (m, n)) if with_add else None
    g = Guarded((m, n), torch.bfloat16)
    y = pk.pact_linear_fp8_fwd(x, w, residual=add, y=g.t)
    pk.pact_check_status()
    g.check()
    check_product(y, x, w, add)
    again = pk.pact_linear_fp8_fwd(x, w, residual=add)
    assert torch.equal(again, y)  # the same bits on every call


@pytest.mark.parametrize("m,n,k", [(4500, 2544, 4112), (8200, 2048, 4240), (5000, 4112, 2064)])
@pytest.mark.parametrize("with_add", [False, True])
def test_linear_many_tiles(m, n, k, with_add):
    """Several waves of tiles, the last of them ragged, against a 64-bit product on the GPU
    with the bound of the other products."""
    rng = np.random.default_rng(m + n)
    g = torch.Generator(device="cuda").manual_seed(m)
    xq = pk.pact_quant_fp8(torch.randn(m, k, device="cuda", generator=g).bfloat16())
    w = random_weight(rng, n, k)
    add = bf16(rng, (m, n)) if with_add else None
    gy = Guarded((m, n), torch.bfloat16)
    y = pk.pact_linear_fp8_fwd(xq, w, residual=add, y=gy.t)
    pk.pact_check_status()
    gy.check()
    a = xq.q.double() * xq.s.double().t().repeat_interleave(128, 1)[:, :k]
    sw = w.s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    b = w.q.double() * sw
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    if add is not None:
        want, mag = want + add.double(), mag + add.double().abs()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -23 * (136 + ref.blocks_of(k)) * mag
    assert bool(((y.double() - want).abs() <= tol * (1 + 2.0 ** -8)).all())
    assert torch.equal(pk.pact_linear_fp8_fwd(xq, w, residual=add), y)


@pytest.mark.parametrize("m,n,k", [(1, 2048, 1024), (12, 528, 4112), (24, 1040, 272), (64, 2048, 2064),
                                   (64, 4096, 2064), (333, 2064, 1040), (640, 1024, 512), (2100, 4080, 528)])
def test_linear_exact_sums(m, n, k):
    """Small whole numbers: every partial sum is exact, so the result is too."""
    rng = np.random.default_rng(k)
    x = torch.from_numpy(rng.integers(-3, 4, (m, k)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.integers(-3, 4, (n, k)).astype(np.float32)).cuda()
    xq = FP8(x.to(torch.float8_e4m3fn), torch.ones(FP8.scale_shape(m, k), device="cuda"))
    wq = FP8Weight(w.to(torch.float8_e4m3fn), torch.ones(FP8Weight.scale_shape(n, k), device="cuda"))
    # powers of two as scales, another for each block
    xq.s *= torch.exp2(torch.from_numpy(rng.integers(-2, 3, xq.s.shape)).cuda())
    wq.s *= torch.exp2(torch.from_numpy(rng.integers(-2, 3, wq.s.shape)).cuda())
    want = ref.dequant(host(xq.q), host(xq.s)) @ ref.dequant_weight(host(wq.q), host(wq.s)).T
    y = pk.pact_linear_fp8_fwd(xq, wq)
    assert torch.equal(y.cpu(), torch.from_numpy(want).float().bfloat16())


@pytest.mark.parametrize("m,n,k", [(1, 1040, 2048), (19, 2048, 512), (333, 1040, 2064),
                                   (515, 2048, 1040)])
def test_linear_dgrad(m, n, k):
    """dX = dY W on the backward layout, added to a gradient in place."""
    rng = np.random.default_rng(m * n + k)
    w = torch.from_numpy((rng.standard_normal((n, k)) * 0.02).astype(np.float32)).cuda()
    wf, wb = pk.pact_pack_weight_fp8_fwd(w), pk.pact_pack_weight_fp8_bwd(w)
    dy = bf16(rng, (m, n), 1e-2)
    if m > 1:
        dy[m // 2] = 0.0
    dyq = pk.pact_quant_fp8(dy)
    prev = bf16(rng, (m, k), 1e-2)
    dx = pk.pact_linear_fp8_dgrad(dyq, wb, dx_prev=prev)
    check_product(dx, dyq, wb, prev)
    # against the formula with the forward layout: dY W
    a, b = ref.dequant(host(dyq.q), host(dyq.s)), ref.dequant_weight(host(wf.q), host(wf.s))
    want = a @ b + host(prev)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -23 * (136 + ref.blocks_of(n)) * (
        np.abs(a) @ np.abs(b) + np.abs(host(prev)))
    assert np.all(np.abs(host(dx) - want) <= tol * (1 + 2.0 ** -8))
    inplace = prev.clone()
    pk.pact_linear_fp8_dgrad(dyq, wb, dx_prev=inplace, dx=inplace)
    assert torch.equal(inplace, dx)
    if m > 1:
        assert torch.equal(pk.pact_linear_fp8_dgrad(dyq, wb)[m // 2],
                           torch.zeros(k, dtype=torch.bfloat16, device="cuda"))


def test_linear_adjoint():
    """<fwd(X), dY> equals <X, dgrad(dY)>: the two layouts hold one weight."""
    rng = np.random.default_rng(77)
    m, n, k = 150, 1040, 784
    lin = Fp8Linear(torch.from_numpy((rng.standard_normal((n, k)) * 0.02).astype(np.float32)).cuda())
    xq, dyq = random_fp8(rng, m, k), random_fp8(rng, m, n)
    y = pk.pact_linear_fp8_fwd(xq, lin.w_fwd)
    dx = pk.pact_linear_fp8_dgrad(dyq, lin.w_bwd)
    x, dy = ref.dequant(host(xq.q), host(xq.s)), ref.dequant(host(dyq.q), host(dyq.s))
    tol = 2.0 ** -8 * (np.abs(host(y) * dy).sum() + np.abs(host(dx) * x).sum())
    assert abs((host(y) * dy).sum() - (host(dx) * x).sum()) <= tol


@pytest.mark.parametrize("m", [1, 5, 40, 300, 1500])
def test_rows_do_not_depend_on_the_batch(m):
    """A token's output is within the product's bound whatever stands beside it, and
    an infinite scale in one row reaches no other."""
    rng = np.random.default_rng(m)
    x, w = random_fp8(rng, m, 1040), random_weight(rng, 528, 1040)
    base = pk.pact_linear_fp8_fwd(x, w)
    if m == 1:
        return
    x.s[:, m // 2] = float("inf")
    y = pk.pact_linear_fp8_fwd(x, w)
    keep = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(y[keep], base[keep])
    assert not bool(torch.isfinite(y[m // 2]).any())


@pytest.mark.parametrize("m,n,k", [(5, 528, 1040), (40, 528, 1040), (700, 528, 4112)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nan_and_infinity_stay_in_their_row(m, n, k, bad):
    rng = np.random.default_rng(m)
    x, w = activation(rng, m, k), random_weight(rng, n, k)
    gamma = bf16(rng, (k,), 0.1) + 1
    quant, norm = pk.pact_quant_fp8(x), pk.pact_add_rmsnorm_quant_fp8(x, None, gamma)[1]
    y, yn = pk.pact_linear_fp8_fwd(quant, w), pk.pact_linear_fp8_fwd(norm, w)
    row = m // 2
    x[row, k - 3] = bad
    keep = torch.arange(m, device="cuda") != row
    for before, made in ((y, pk.pact_quant_fp8(x)),
                         (yn, pk.pact_add_rmsnorm_quant_fp8(x, None, gamma)[1])):
        assert bool(torch.isnan(made.q[row, k - 3].float()))
        after = pk.pact_linear_fp8_fwd(made, w)
        assert torch.equal(after[keep], before[keep])
        assert bool(torch.isnan(after[row]).all())


@pytest.mark.parametrize("m,h", [(300, 1040), (2, 16384), (3, 64), (5000, 1040), (600, 16384)])
def test_add_rmsnorm_bwd_over_h(m, h):
    """dh written over h gives what it gives elsewhere."""
    rng = np.random.default_rng(m + h)
    hh, dy, gamma = bf16(rng, (m, h)), bf16(rng, (m, h)), bf16(rng, (h,))
    rstd = pk.pact_add_rmsnorm_quant_fp8(hh, None, gamma)[2]
    dh, dg = pk.pact_add_rmsnorm_bwd(hh, gamma, rstd, dy, dgamma=True)
    got, dg2 = pk.pact_add_rmsnorm_bwd(hh, gamma, rstd, dy, dh=hh, dgamma=True)
    assert got is hh and torch.equal(got, dh)
    assert torch.equal(dg2, dg)


def test_product_offsets_past_32_bits():
    """An input and an output of more than 2^32 values: the rows at the end are those
    of a small call on them."""
    m, n, k = 270000, 16384, 16384
    rng = np.random.default_rng(2)
    xq = FP8(torch.zeros((m, k), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
             torch.ones(FP8.scale_shape(m, k), device="cuda"))
    w = random_weight(rng, n, k)
    tail = random_fp8(rng, 300, k)
    xq.q.view(torch.uint8)[-300:] = tail.q.view(torch.uint8)
    xq.s[:, -300:] = tail.s
    y = pk.pact_linear_fp8_fwd(xq, w)
    assert not bool(y[:-300:997].any())
    a, b = ref.dequant(host(tail.q)[-4:], host(tail.s)[:, -4:]), ref.dequant_weight(host(w.q), host(w.s))
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -23 * (128 + 128 + 8) * mag
    assert np.all(np.abs(host(y[-4:]) - want) <= tol * (1 + 2.0 ** -8))


# ---------------------------------------------------------------- as they are used
def _block(m, hidden, inter, seed):
    """norm -> linear (up) -> quant -> linear (down, with the residual), and back."""
    rng = np.random.default_rng(seed)
    up = Fp8Linear(torch.from_numpy((rng.standard_normal((inter, hidden)) * 0.02).astype(np.float32)).cuda())
    down = Fp8Linear(torch.from_numpy((rng.standard_normal((hidden, inter)) * 0.02).astype(np.float32)).cuda())
    d = dict(x=bf16(rng, (m, hidden)), res=bf16(rng, (m, hidden)), dy=bf16(rng, (m, hidden), 1e-2),
             gamma=(1 + bf16(rng, (hidden,), 0.1)).bfloat16())
    return up, down, d


def _run(up, down, d):
    h, hq, rstd = pk.pact_add_rmsnorm_quant_fp8(d["x"], d["res"], d["gamma"])
    a = up.forward(hq)
    aq = pk.pact_quant_fp8(a)
    out = down.forward(aq, residual=h)
    da = down.dgrad(d["dy"])
    dn = up.dgrad(da)
    dh, dgamma = pk.pact_add_rmsnorm_bwd(h, d["gamma"], rstd, dn, dres=d["dy"], dgamma=True)
    return dict(h=h, hq=hq.q, hs=hq.s, rstd=rstd, a=a, aq=aq.q, as_=aq.s, out=out, da=da, dn=dn,
                dh=dh, dgamma=dgamma)


@pytest.mark.parametrize("m", [1, 20, 333])
def test_block_forward_and_backward(m):
    up, down, d = _block(m, 528, 1040, m)
    r = _run(up, down, d)
    pk.pact_check_status()
    hq, aq = FP8(r["hq"], r["hs"]), FP8(r["aq"], r["as_"])
    assert torch.equal(r["h"], (d["x"].float() + d["res"].float()).bfloat16())
    check_product(r["a"], hq, up.w_fwd)
    assert_fp8_bits(aq, *ref.quant_fp32(r["a"].float().cpu().numpy()))
    check_product(r["out"], aq, down.w_fwd, r["h"])
    check_product(r["da"], pk.pact_quant_fp8(d["dy"]), down.w_bwd)
    check_product(r["dn"], pk.pact_quant_fp8(r["da"]), up.w_bwd)
    want, want_g, mags = ref.norm_bwd(host(r["h"]), host(d["gamma"]), host(r["rstd"]), host(r["dn"]),
                                      host(d["dy"]))
    tol = 2.0 ** -8 * np.abs(want) + U * (4 * mags[0] + 8 * mags[1] * mags[2]
                                          + 64 * mags[1] * mags[3] + np.abs(host(d["dy"])))
    assert np.all(np.abs(host(r["dh"]) - want) <= tol * (1 + 2.0 ** -8))
    assert np.all(np.abs(host(r["dgamma"]) - want_g) <= U * (80 + m) * mags[4])


def test_on_another_stream():
    up, down, d = _block(40, 1040, 2064, 1)
    want = _run(up, down, d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _run(up, down, d)
    side.synchronize()
    for k in want:
        assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), k


def test_two_captured_graphs_replayed_side_by_side():
    """Each graph keeps scratch of its own: replayed at once on two streams, again and
    again, both give what eager calls give; new inputs in the same buffers count."""
    sets = [_block(m, 1040, 2064, 10 + m) for m in (600, 24)]
    eager = [_run(*s) for s in sets]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_run(*s))
        graphs.append(g)
    for turn in range(3):
        for st, g in zip(streams, graphs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for want, got in zip(eager, outs):
            for k in want:
                assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), (turn, k)
        if turn == 1:
            for s in sets:
                s[2]["x"].copy_(s[2]["x"].flip(0) * 2)
            eager = [_run(*s) for s in sets]
            torch.cuda.synchronize()
    pk.pact_check_status()


# ---------------------------------------------------------------- refusals
def test_python_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    q, w = pk.pact_quant_fp8(x), pk.pact_pack_weight_fp8_fwd(torch.zeros((32, 64), device="cuda"))
    gamma, rstd = torch.ones(64, dtype=torch.bfloat16, device="cuda"), torch.ones(4, device="cuda")
    y = torch.empty((4, 32), dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: pk.pact_quant_fp8(x.float()),
        lambda: pk.pact_quant_fp8(x.t()),
        lambda: pk.pact_quant_fp8(x, out=FP8.empty(4, 48)),
        lambda: pk.pact_quant_fp8(x, out=FP8Weight.empty(4, 64)),
        lambda: pk.pact_quant_fp8(x, out=FP8(q.q, q.s.t())),
        lambda: pk.pact_pack_weight_fp8_fwd(x),
        lambda: pk.pact_linear_fp8_fwd(w, w),
        lambda: pk.pact_linear_fp8_fwd(q, q),
        lambda: pk.pact_linear_fp8_fwd(q, FP8Weight.empty(32, 48)),
        lambda: pk.pact_linear_fp8_fwd(q, w, y=y.float()),
        lambda: pk.pact_linear_fp8_fwd(q, w, y=y[:, :16]),
        lambda: pk.pact_linear_fp8_fwd(q, w, residual=x),
        lambda: pk.pact_linear_fp8_fwd(FP8(q.q.view(torch.uint8), q.s), w),
        lambda: pk.pact_add_rmsnorm_quant_fp8(x, x[:2], gamma),
        lambda: pk.pact_add_rmsnorm_quant_fp8(x, x, gamma[:32]),
        lambda: pk.pact_add_rmsnorm_quant_fp8(x, None, gamma, h=torch.empty_like(x)),
        lambda: pk.pact_add_rmsnorm_quant_fp8(x, x.t().contiguous().t(), gamma),
        lambda: pk.pact_add_rmsnorm_bwd(x, gamma, rstd[:3], x),
        lambda: pk.pact_add_rmsnorm_bwd(x, gamma, rstd, x, dgamma=gamma),
        lambda: pk.pact_add_rmsnorm_bwd(x, gamma, rstd, x.float()),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was accepted")


def test_library_refusals():
    """Shapes that pass the binding and that the library refuses before any launch."""
    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    before = pk.pact_launch_count()
    bad = [
        (2, lambda: pk.pact_quant_fp8(z(4, 24))),
        (2, lambda: pk.pact_quant_fp8(z(0, 64))),
        (2, lambda: pk.pact_quant_fp8(z(4, 68)[:, :64])),
        (3, lambda: pk.pact_quant_fp8(z(4, 136)[:, 4:132])),
        (2, lambda: pk.pact_pack_weight_fp8_fwd(z(24, 64, dtype=torch.float32))),
        (2, lambda: pk.pact_linear_fp8_fwd(FP8.empty(0, 64), FP8Weight.empty(32, 64))),
        (2, lambda: pk.pact_linear_fp8_fwd(FP8.empty(4, 72), FP8Weight.empty(32, 72))),
        (2, lambda: pk.pact_linear_fp8_fwd(FP8.empty(4, 64), FP8Weight.empty(40, 64))),
        (2, lambda: pk.pact_add_rmsnorm_quant_fp8(z(4, 40), None, z(40))),
        (2, lambda: pk.pact_add_rmsnorm_quant_fp8(z(1, 16400), None, z(16400))),
        (1, lambda: pk.pact_add_rmsnorm_quant_fp8(z(4, 64), None, z(64), eps=-1.0)),
        (1, lambda: pk.pact_add_rmsnorm_quant_fp8(z(4, 64), None, z(64), eps=float("nan"))),
        (3, lambda: pk.pact_add_rmsnorm_quant_fp8(z(257)[1:].view(4, 64), None, z(64))),
        (2, lambda: pk.pact_add_rmsnorm_bwd(z(0, 64), z(64), z(0, dtype=torch.float32), z(0, 64))),
    ]
    for k, (code, call) in enumerate(bad):
        with pytest.raises(pk.PactError) as e:
            call()
            pytest.fail(f"call {k} was accepted")
        assert e.value.code == code, (k, str(e.value))
    assert pk.pact_launch_count() == before
