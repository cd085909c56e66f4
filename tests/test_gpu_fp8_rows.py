"""What a row of the FP8 calls depends on, and dgamma's bound by the kernel's own order of
sums.

dgamma (u = 2^-24): a group of warps adds its rows in a chain of fused steps, one partial
row a group; 64 lanes then add ceil(partial rows / 64) of them each, and 7 + 7 joins follow.
With n = RN(h rstd) a term carries u of its own:
  u (rows of a group + ceil(partial rows / 64) + 14 + 2) sum |dy n|
The groups, from the widths: up to 256 columns 8 a CTA and three CTAs an SM, wider ones
fewer; above 4096 columns one an SM.
"""
import pytest
import torch

import fp8_paths
import nvfp4_frozen_projection_gb300 as pk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _groups(h):
    """Groups of warps in flight on a full grid of the norm's backward (152 SMs)."""
    per_warp = 1024 if h > 8192 else 512
    wpr = 1
    while h > wpr * per_warp:
        wpr *= 2
    if wpr > 8:
        return 152
    return 152 * (3 if h <= wpr * 256 else 2) * (8 // wpr)


@pytest.mark.parametrize("m,h", [(30000, 8192), (40000, 256), (60000, 1040), (20000, 12304),
                                 (25000, 4096)])
def test_dgamma_of_many_rows(m, h):
    g = torch.Generator(device="cuda").manual_seed(m + h)
    x = torch.randn(m, h, device="cuda", generator=g).bfloat16()
    dy = (0.01 * torch.randn(m, h, device="cuda", generator=g)).bfloat16()
    gamma = (1 + 0.1 * torch.randn(h, device="cuda", generator=g)).bfloat16()
    rstd = pk.pact_add_rmsnorm_quant_fp8(x, None, gamma)[2]
    assert pk.load_library().pact_add_rmsnorm_bwd_workspace_size(m, h) == -(-_groups(h) * h * 4 // 256) * 256
    _, dgamma = pk.pact_add_rmsnorm_bwd(x, gamma, rstd, dy, dgamma=True)
    pk.pact_check_status()
    terms = dy.double()
    terms *= x.double()
    terms *= rstd.double()[:, None]
    want, mag = terms.sum(0), terms.abs().sum(0)
    chain = -(-m // _groups(h)) + -(-_groups(h) // 64) + 14 + 2
    over = (dgamma.double() - want).abs() - U * chain * mag * (1 + 2.0 ** -8)
    assert bool((over <= 0).all()), float(over.max())


@pytest.mark.parametrize("m,n,k", [s for s in fp8_paths.SHAPES if s[0] > 1])
def test_a_products_row_does_not_depend_on_its_neighbours(m, n, k):
    """Other rows beside it: the same bits.  Alone: within the product's bound."""
    g = torch.Generator(device="cuda").manual_seed(m * n + k)
    row = m // 3
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    other = (30 * torch.randn(m, k, device="cuda", generator=g)).bfloat16()
    other[row] = x[row]
    other[(row + 1) % m] = 0.0
    w = pk.pact_pack_weight_fp8_fwd(0.02 * torch.randn(n, k, device="cuda", generator=g))
    xq = pk.pact_quant_fp8(x)
    y = pk.pact_linear_fp8_fwd(xq, w)[row].clone()
    assert torch.equal(pk.pact_linear_fp8_fwd(pk.pact_quant_fp8(other), w)[row], y)
    alone = pk.pact_linear_fp8_fwd(pk.pact_quant_fp8(x[row:row + 1]), w)[0]
    pk.pact_check_status()
    a = xq.q[row].double() * xq.s[:, row].double().repeat_interleave(128)[:k]
    s = w.s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    b = w.q.double() * s
    want, mag = b @ a, b.abs() @ a.abs()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -23 * (136 + -(-k // 128)) * mag
    for got in (y, alone):
        over = (got.double() - want).abs() - tol * (1 + 2.0 ** -8)
        assert bool((over <= 0).all()), float(over.max())


@pytest.mark.parametrize("m,h", [(2, 2048), (9, 256), (333, 1040), (700, 8192), (300, 12304)])
def test_a_norms_row_does_not_depend_on_its_neighbours(m, h):
    g = torch.Generator(device="cuda").manual_seed(m + h)
    row = m // 3
    x, res, dy, o1, o2, o3 = (torch.randn(m, h, device="cuda", generator=g).bfloat16()
                              for _ in range(6))
    for o, t in ((o1, x), (o2, res), (o3, dy)):
        o *= 5
        o[row] = t[row]
    gamma = (1 + 0.1 * torch.randn(h, device="cuda", generator=g)).bfloat16()
    got = []
    for a, r, d in ((x, res, dy), (o1, o2, o3)):
        hh, yq, rstd = pk.pact_add_rmsnorm_quant_fp8(a, r, gamma)
        dh, _ = pk.pact_add_rmsnorm_bwd(hh, gamma, rstd, d, dres=r, dgamma=True)
        got.append([hh[row], yq.q[row].view(torch.uint8), yq.s[:, row], rstd[row], dh[row]])
    pk.pact_check_status()
    for a, b in zip(*got):
        assert torch.equal(a, b)
